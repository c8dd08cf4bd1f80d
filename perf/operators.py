"""Measured cases of three operators of the library, each in its plain form (elementary torch operations) and,
with ``own`` set, as the calls a user makes of the binding.

  prep   o1_head_prep          per-head norm of queries and keys with the rotary rotation
  chunk  o1_lin_chunk_attend   linear attention with a decay per head over prompts (packed sequences)
  token  o1_lin_token_attend   the same, one row per sequence

Linear attention, head h with decay l = exp(log_decay[h]) and state S [d][dv]:
S_t = l S_{t-1} + k_t v_t^T, o_t = scale q_t S_t.
"""
import math

import torch

own = False

F32, BF16, F16 = "f32", "bf16", "f16"
_TYPES = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}
_BYTES = {F32: 4, BF16: 2, F16: 2}
EPS = 1e-6


def listed():
    return [
        # one decode row of the Qwen3.5-0.8B-shaped layer (8 query and 2 key heads of 256): launch latency
        dict(name="prep one row", op="prep", rows=1, hq=8, hk=2, d=256, rot=256, norm="rms", tin=F32, tout=F32,
             fused=False, pos_max=8192),
        # an odd draft-sized batch of wide heads rotated in part, half precision in, the sealed layer's f32 out
        dict(name="prep partial rotation", op="prep", rows=999, hq=9, hk=3, d=200, rot=56, norm="unit", tin=F16,
             tout=F32, fused=True, pos_max=1 << 20),
        # the 4096-row prompt of the same layer, f32 throughout as the sealed layer takes it
        dict(name="prep prompt", op="prep", rows=4096, hq=8, hk=2, d=256, rot=256, norm="rms", tin=F32, tout=F32,
             fused=False, pos_max=4096),
        # a large mixed batch of the stack layer's heads, read in place from fused q|k|v rows, far positions
        dict(name="prep batch", op="prep", rows=32749, hq=16, hk=4, d=128, rot=128, norm="rms", tin=BF16, tout=BF16,
             fused=True, pos_max=1 << 20),
        # one 64-row chunk of the stack layer: the pages' calling pattern
        dict(name="chunk 64 rows", op="chunk", lens="64", slots=1, groups=4, hpg=4, d=128, dv=128, t=F32),
        # odd widths and heads, half precision
        dict(name="chunk odd widths", op="chunk", lens="1000,77", slots=3, groups=3, hpg=1, d=72, dv=40, t=F16),
        # a ragged batch of prompts of the stack layer, one empty and one of a single row among them
        dict(name="chunk ragged", op="chunk", lens="700,1,2047,0,130,1500,17,64,333", slots=12, groups=4, hpg=4,
             d=128, dv=128, t=BF16),
        # the 4096-row prompt of the Qwen3.5-0.8B-shaped layer
        dict(name="chunk prompt", op="chunk", lens="4096", slots=1, groups=2, hpg=4, d=256, dv=256, t=F32),
        # the 32768-row prompt
        dict(name="chunk long prompt", op="chunk", lens="32768", slots=1, groups=2, hpg=4, d=256, dv=256, t=BF16),
        # one decode step of one sequence
        dict(name="token one", op="token", rows=1, slots=1, pad=0, groups=2, hpg=4, d=256, dv=256, t=F32),
        # a decode batch of the stack layer, some rows padding
        dict(name="token batch", op="token", rows=61, slots=80, pad=3, groups=4, hpg=4, d=128, dv=128, t=BF16),
        # a large decode batch: 0.5 GB of state read and written
        dict(name="token large", op="token", rows=512, slots=512, pad=0, groups=4, hpg=4, d=128, dv=128, t=F32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "chunk", "chunk", "token"])
    if op == "prep":
        d = 8 * rng.randint(4, 32)
        rot = d if d % 16 == 0 and rng.random() < 0.5 else 8 * rng.randint(0, d // 8)
        tin = rng.choice([F32, BF16, F16])
        return dict(op=op, rows=_log(rng, 1, 16000), hq=rng.randint(1, 16), hk=rng.randint(1, 8), d=d, rot=rot,
                    norm=rng.choice(["rms", "unit", "none"]), tin=tin, tout=rng.choice([tin, F32]),
                    fused=rng.random() < 0.5, pos_max=_log(rng, 64, 1 << 24))
    groups, hpg = rng.randint(1, 4), rng.randint(1, 4)
    d, dv = rng.choice([(64, 64), (128, 128), (256, 256), (8 * rng.randint(2, 32), 8 * rng.randint(2, 32))])
    t = rng.choice([F32, BF16, F16])
    if op == "chunk":
        n = rng.randint(1, 6)
        lens = [rng.choice([0, 1, _log(rng, 2, 4096), _log(rng, 2, 4096), _log(rng, 2, 4096)]) for _ in range(n)]
        lens.append(_log(rng, 2, 4096))
        return dict(op=op, lens=",".join(map(str, lens)), slots=len(lens) + rng.randint(0, 3), groups=groups, hpg=hpg,
                    d=d, dv=dv, t=t)
    rows = _log(rng, 1, 128)
    pad = rng.randint(0, rows // 4)
    return dict(op=op, rows=rows, slots=rows + rng.randint(0, 9), pad=pad, groups=groups, hpg=hpg, d=d, dv=dv, t=t)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    s = dict(case=case)
    if case["op"] == "prep":
        rows, hq, hk, d, rot = (case[k] for k in ("rows", "hq", "hk", "d", "rot"))
        tin, tout = _TYPES[case["tin"]], _TYPES[case["tout"]]
        if case["fused"]:
            # q, k and a value part side by side in one projection's rows
            x = randn(rows, (hq + 2 * hk) * d, dtype=tin)
            s["q"] = x[:, :hq * d].unflatten(1, (hq, d))
            s["k"] = x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        else:
            s["q"], s["k"] = randn(rows, hq, d, dtype=tin), randn(rows, hk, d, dtype=tin)
        s["wq"], s["wk"] = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
        j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
        s["inv"] = (1e6 ** (-2.0 * j / max(rot, 1))).float()
        s["pos"] = torch.randint(0, case["pos_max"], (rows,), generator=gen, device="cuda")
        s["q_out"] = torch.zeros(rows, hq, d, dtype=tout, device="cuda")
        s["k_out"] = torch.zeros(rows, hk, d, dtype=tout, device="cuda")
        return s
    groups, hpg, d, dv, t = case["groups"], case["hpg"], case["d"], case["dv"], _TYPES[case["t"]]
    nh, slots = groups * hpg, case["slots"]
    # decays from fast to slow heads, and a state of the size that such a decay leaves
    h = torch.arange(nh, device="cuda", dtype=torch.float32)
    s["g"] = -torch.exp2(1.0 - 11.0 * (h + torch.rand(nh, generator=gen, device="cuda")) / nh)
    s["state"] = randn(slots, nh, d, dv) / (-torch.expm1(2 * s["g"])).sqrt().view(1, nh, 1, 1)
    if case["op"] == "chunk":
        lens = _lens(case)
        rows = sum(lens) + 5 * (len(lens) > 1)   # a few rows of no sequence at the end
        order = torch.randperm(slots, generator=gen, device="cuda")[:len(lens)].tolist()
        starts = [sum(lens[:i]) for i in range(len(lens))]
        s["seqs"] = list(zip(starts, lens, order))
        chunks = sum((n + 63) // 64 for n in lens) + len(lens)
        s["scratch"] = torch.empty(chunks * nh * d * dv * 4 + (1 << 20), dtype=torch.uint8, device="cuda")
    else:
        rows = case["rows"]
        idx = torch.randperm(slots, generator=gen, device="cuda")[:rows].to(torch.int32)
        if case["pad"]:
            idx[torch.randperm(rows, generator=gen, device="cuda")[:case["pad"]]] = -1
        s["slots"] = idx
    s["q"], s["k"], s["v"] = randn(rows, nh, d, dtype=t), randn(rows, groups, d, dtype=t), randn(rows, groups, dv, dtype=t)
    s["out"] = torch.zeros(rows, nh, dv, dtype=t, device="cuda")
    return s


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"prep": _prep, "chunk": _chunk, "token": _token}[case["op"]](s, case)


def _own(s, case):
    from sliding_window_landmark_gb300 import o1
    if case["op"] == "prep":
        if "geom" not in s:
            s["geom"] = o1.prep_geom(case["hq"], case["hk"], case["d"], rot=case["rot"], norm=case["norm"],
                                     in_dtype=s["q"].dtype, out_dtype=s["q_out"].dtype, eps=EPS)
        o1.check(o1.o1_head_prep(s["geom"], s["q"], s["k"], s["wq"], s["wk"], s["inv"], s["q_out"], s["k_out"],
                                 pos=s["pos"]), "prep")
        return s["q_out"], s["k_out"]
    if "geom" not in s:
        s["geom"] = o1.lin_geom(case["groups"], case["hpg"], case["d"], case["dv"], dtype=s["q"].dtype)
        if case["op"] == "chunk":
            # the scratch as a user's program sizes it: by the library's own function
            s["scratch"] = torch.empty(o1.o1_lin_scratch_bytes(s["geom"], s["q"].shape[0], len(s["seqs"])),
                                       dtype=torch.uint8, device="cuda")
    if case["op"] == "chunk":
        o1.check(o1.o1_lin_chunk_attend(s["state"], s["geom"], s["scratch"], s["q"], s["k"], s["v"], s["g"],
                                        s["seqs"], s["out"]), "chunk")
    else:
        o1.check(o1.o1_lin_token_attend(s["state"], s["geom"], s["q"], s["k"], s["v"], s["g"], s["slots"],
                                        s["out"]), "token")
    return s["out"], s["state"]


# ------------------------------------------------------------ plain forms

def _normed(x, w, norm):
    x = x.float()
    if norm == "rms":
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    elif norm == "unit":
        x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)
    return x * w


def _prep(s, case):
    half = case["rot"] // 2
    a = s["pos"].double()[:, None] * s["inv"].double()   # angles of far positions: 64 bits
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    res = []
    for x, w, out in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
        y = _normed(x, w, case["norm"])
        y0, y1 = y[..., :half], y[..., half:2 * half]
        out.copy_(torch.cat([y0 * cos - y1 * sin, y1 * cos + y0 * sin, y[..., 2 * half:]], -1))
        res.append(out)
    return tuple(res)


def _powers(g, n):
    """exp(g n), g [nh] per head on the leading axis; 0 where n < 0. The exponent in 64 bits."""
    n = n.double()
    e = torch.exp(g.double().view(-1, *[1] * n.dim()) * n.clamp(min=0))
    return torch.where(n >= 0, e, torch.zeros_like(e)).float()


def _chunk(s, case):
    """All sequences padded to one length and cut into chunks of C rows: the causal products inside each chunk, the
    chunks' state increments, and their decayed sums as one product over the chunks."""
    C, hpg, d, dv, g = 128, case["hpg"], case["d"], case["dv"], s["g"]
    nh, scale = g.numel(), 1.0 / math.sqrt(d)
    row0, rows, slot = torch.tensor(s["seqs"], device="cuda").T
    B, nc = row0.numel(), max(1, -(-max(n for _, n, _ in s["seqs"]) // C))
    t = torch.arange(nc * C, device="cuda")
    valid = t < rows[:, None]                                                          # [B, L]
    at = torch.where(valid, row0[:, None] + t, 0)

    def lay(x, heads):   # [B, nh, nc, C, width], zero past the sequence's end
        x = torch.where(valid[..., None, None], x[at].float(), 0.0)
        return x.repeat_interleave(heads, 2).permute(0, 2, 1, 3).unflatten(2, (nc, C))

    q, k, v = lay(s["q"], 1), lay(s["k"], hpg), lay(s["v"], hpg)
    i, c = torch.arange(C, device="cuda"), torch.arange(nc, device="cuda")
    S0 = s["state"][slot]                                                               # [B, nh, d, dv]
    p = (q @ k.transpose(-1, -2)) * _powers(g, i[:, None] - i)[:, None]
    o = p @ v
    inc = ((k * _powers(g, C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v).flatten(-2)   # [B, nh, nc, d dv]
    enter = _powers(g, C * (c[:, None] - 1 - c)) @ inc + _powers(g, C * c)[..., None] * S0.flatten(-2)[:, :, None]
    o = o + _powers(g, i + 1)[:, None, :, None] * (q @ enter.unflatten(-1, (d, dv)))
    o = (o * scale).flatten(2, 3).transpose(1, 2)                                       # [B, L, nh, dv]
    s["out"][at[valid]] = o[valid].to(s["out"].dtype)
    w = _powers(g, rows[:, None] - 1 - t).transpose(0, 1)[..., None]                    # [B, nh, L, 1]
    last = (k.flatten(2, 3) * w).transpose(-1, -2) @ v.flatten(2, 3)
    s["state"][slot] = last + _powers(g, rows).T[..., None, None] * S0
    return s["out"], s["state"]


def _token(s, case):
    hpg, scale = case["hpg"], 1.0 / math.sqrt(case["d"])
    live = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][live].long()
    q, k, v = (s[n][live].float() for n in "qkv")
    k, v = k.repeat_interleave(hpg, 1), v.repeat_interleave(hpg, 1)
    S = s["state"][slot] * s["g"].exp().view(1, -1, 1, 1) + k[..., :, None] * v[..., None, :]
    s["state"][slot] = S
    s["out"][live] = ((q[..., None, :] @ S)[..., 0, :] * scale).to(s["out"].dtype)
    return s["out"], s["state"]


# ------------------------------------------------------------ cost and truth

def work(case):
    if case["op"] == "prep":
        n = case["rows"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": n * (_BYTES[case["tin"]] + _BYTES[case["tout"]]) + 8 * case["rows"] + 8 * case["d"]
                + 2 * case["rot"], "flops": 8 * n}
    groups, d, dv, b = case["groups"], case["d"], case["dv"], _BYTES[case["t"]]
    nh = groups * case["hpg"]
    if case["op"] == "chunk":
        lens = _lens(case)
        rows, live = sum(lens), sum(n > 0 for n in lens)
    else:
        rows = live = case["rows"] - case["pad"]
    # every row's q, k, v and output once, every touched state read and written once; the recurrence's products
    return {"bytes": rows * (nh * (d + dv) + groups * (d + dv)) * b + live * nh * d * dv * 8 + 4 * nh,
            "flops": 4 * rows * nh * d * dv}


def _exact_prep(s, case):
    res = []
    a = s["pos"].double()[:, None, None] * s["inv"].double()
    h = case["rot"] // 2
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        n2 = x.pow(2).sum(-1, keepdim=True)
        r = {"rms": (n2 / case["d"] + EPS).rsqrt(), "unit": (n2 + EPS).rsqrt(), "none": torch.ones_like(n2)}[case["norm"]]
        y = x * r * w.double()
        z = torch.complex(y[..., :h], y[..., h:2 * h]) * torch.polar(torch.ones_like(a), a)
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
        res.append(y)
    return tuple(res)


def exact(case, seed):
    """The definitions in 64 bits: the rotation as a complex product; the recurrence one row at a time."""
    s = prepare(case, seed)
    if case["op"] == "prep":
        return _exact_prep(s, case)
    hpg, scale = case["hpg"], 1.0 / math.sqrt(case["d"])
    lam = s["g"].double().exp().view(-1, 1, 1)
    out, state = s["out"].double(), s["state"].double()
    seqs = s["seqs"] if case["op"] == "chunk" else [(r, 1, i) for r, i in enumerate(s["slots"].tolist()) if i >= 0]
    for row0, rows, slot in seqs:
        S = state[slot]                                                        # a view, advanced in place
        q = s["q"][row0:row0 + rows].double().unsqueeze(2) * scale             # [n, nh, 1, d]
        k = s["k"][row0:row0 + rows].double().repeat_interleave(hpg, 1).unsqueeze(3)
        v = s["v"][row0:row0 + rows].double().repeat_interleave(hpg, 1).unsqueeze(2)
        for r in range(rows):
            S.mul_(lam).addcmul_(k[r], v[r])
            out[row0 + r] = torch.matmul(q[r], S)[:, 0]
    return out, state
