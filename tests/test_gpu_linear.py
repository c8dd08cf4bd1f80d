"""The linear layer on the GPU (o1_lin_chunk_attend, o1_lin_token_attend)
against the 64-bit row-by-row reference, held to the bounds derived in
lin_reference: chunk boundaries, lengths of zero and one, packed batches,
head layouts, odd widths, element types, strides, decays of 0 and -inf,
padding, rows and slots left alone, passes of a small scratch, capture and
replay, other streams."""
import pytest
import torch

import lin_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def o1():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_landmark_gb300 import build
    build.build()
    from sliding_window_landmark_gb300 import o1 as mod
    return mod


def make(groups, hpg, d, dv, rows, slots, dtype, seed, decay=None):
    gen = torch.Generator().manual_seed(seed)
    nh = groups * hpg
    t = lambda *s: torch.randn(*s, generator=gen)
    x = dict(q=t(rows, nh, d).to(dtype), k=t(rows, groups, d).to(dtype), v=t(rows, groups, dv).to(dtype),
             state=3 * t(slots, nh, d, dv), g=-torch.exp2(1 - 9 * torch.rand(nh, generator=gen)))
    if decay is not None:
        x["g"] = torch.tensor([decay[i % len(decay)] for i in range(nh)], dtype=F32)
    return {n: v.cuda() for n, v in x.items()}


def chunk(o1, x, geom, seqs, out, scratch_rows=None, stream=None):
    rows = x["q"].shape[0]
    nbytes = o1.o1_lin_scratch_bytes(geom, scratch_rows or max(rows, 1), 1 if scratch_rows else max(1, len(seqs)))
    scratch = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    o1.check(o1.o1_lin_chunk_attend(x["state"], geom, scratch, x["q"], x["k"], x["v"], x["g"], seqs, out, stream=stream),
             "chunk")
    return scratch


def check(o1, x, state0, seqs, out, scale, what):
    want, Ao, S, As = ref.linear(x["q"], x["k"], x["v"], x["g"], state0, seqs, scale)
    bo, bs = ref.linear_bounds(want, Ao, As, seqs, x["q"].dtype)
    live = torch.zeros(want.shape[0], dtype=torch.bool)
    for r0, n, _ in seqs:
        live[r0:r0 + n] = True
    ref.assert_within(out[live.to(out.device)], want[live], bo[live], what + " out")
    # slots of no sequence have a bound of 0: bit for bit as they were
    ref.assert_within(x["state"], S, bs, what + " state")
    assert torch.isnan(out[~live.to(out.device)]).all(), what + ": rows of no sequence were written"


# groups, heads per group, d, dv, [lengths], dtype, decays (None: spread)
CASES = [
    (1, 1, 64, 64, [1], F32, None),
    (1, 2, 64, 64, [2], BF16, None),
    (2, 1, 64, 64, [64], F32, None),
    (2, 2, 128, 128, [65], BF16, None),
    (1, 2, 64, 64, [127], F16, None),
    (1, 2, 128, 64, [128], F32, None),
    (2, 2, 64, 128, [129], BF16, None),
    (2, 4, 256, 256, [200], F32, None),
    (1, 4, 256, 256, [300], BF16, None),
    (1, 1, 8, 8, [140], F32, None),
    (1, 3, 8, 256, [70], BF16, None),
    (3, 1, 256, 8, [131], F16, None),
    (3, 1, 72, 40, [150, 77], F16, None),
    (1, 2, 200, 136, [90, 140], F32, None),
    (4, 4, 128, 128, [70, 1, 0, 257, 33, 128, 5], BF16, None),
    (2, 2, 64, 64, [0, 0, 3], F32, None),
    (2, 2, 64, 64, [0], F32, None),
    (1, 4, 64, 64, [300], F32, [0.0, -1e-4, float("-inf"), -40.0]),
    (1, 4, 64, 64, [300, 20], BF16, [0.0, -1e-4, float("-inf"), -40.0]),
    (1, 16, 32, 32, [140], BF16, None),
    (5, 1, 96, 96, [513], F32, None),
    (1, 1, 128, 128, [700], F16, None),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_chunk(o1, case):
    G, hpg, d, dv, lens, dt, decay = CASES[case]
    rows, slots = sum(lens) + 3, len(lens) + 2
    x = make(G, hpg, d, dv, rows, slots, dt, 100 + case, decay)
    seqs, r = [], 1
    for i, n in enumerate(lens):   # one row before, two after; slots in an order of their own
        seqs.append((r, n, (2 * i + 1) % slots if slots % 2 else (i + 1) % slots))
        r += n
    for row in [0, r, r + 1]:      # rows of no sequence hold NaN and infinities
        x["q"][row], x["k"][row], x["v"][row] = float("nan"), float("inf"), float("nan")
    geom = o1.lin_geom(G, hpg, d, dv, dtype=dt)
    out = torch.full((rows, G * hpg, dv), float("nan"), dtype=dt, device="cuda")
    state0 = x["state"].clone()
    chunk(o1, x, geom, seqs, out)
    torch.cuda.synchronize()
    check(o1, x, state0, seqs, out, geom.scale, f"case {case}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_many_tiles(o1, dt):
    """More tiles than SMs: segments of 256 rows, of which sequences leave 1 to
    256, and several of them, long and short in turn, for a block of threads."""
    G, hpg, d, dv = 4, 2, 72, 136
    lens = [700, 129, 130, 256, 64, 255, 257, 300, 128, 513, 49, 1025, 384, 100]
    rows = sum(lens) + 2
    x = make(G, hpg, d, dv, rows, len(lens), dt, 61)
    seqs = [(sum(lens[:i]), n, len(lens) - 1 - i) for i, n in enumerate(lens)]
    x["q"][-2:], x["k"][-2:], x["v"][-2:] = float("inf"), float("nan"), float("nan")
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=dt), x["state"].clone()
    out = torch.full((rows, G * hpg, dv), float("nan"), dtype=dt, device="cuda")
    chunk(o1, x, geom, seqs, out)
    torch.cuda.synchronize()
    check(o1, x, s0, seqs, out, geom.scale, f"many tiles {dt}")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("lens", [[300] + 40 * [1] + 3 * [16] + [0, 31, 49], 3 * [2] + [260], 2 * [33] + 30 * [5]])
def test_short_sequences_beside_long_ones(o1, dt, lens):
    """Short sequences by rows or with the tiles, whichever the call takes."""
    G, hpg, d, dv = 2, 4, 64, 128
    rows = sum(lens)
    x = make(G, hpg, d, dv, rows, len(lens), dt, 67)
    seqs = [(sum(lens[:i]), n, len(lens) - 1 - i) for i, n in enumerate(lens)]
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=dt), x["state"].clone()
    out = torch.full((rows, G * hpg, dv), float("nan"), dtype=dt, device="cuda")
    chunk(o1, x, geom, seqs, out)
    torch.cuda.synchronize()
    check(o1, x, s0, seqs, out, geom.scale, f"{len(lens)} sequences {dt}")


@pytest.mark.parametrize("width", [128, 256])
@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_chunk_relative_error(o1, dt, width):
    """In the 2-norm the f32 path and every state are near fp32's own error."""
    x = make(2, 2, width, width, 600, 1, dt, 7)
    geom = o1.lin_geom(2, 2, width, width, dtype=dt)
    out, s0 = torch.empty(600, 4, width, dtype=dt, device="cuda"), x["state"].clone()
    chunk(o1, x, geom, [(0, 600, 0)], out)
    want, _, S, _ = ref.linear(x["q"], x["k"], x["v"], x["g"], s0, [(0, 600, 0)], geom.scale)
    rel = [float((got.cpu().double() - w).norm() / w.norm()) for got, w in ((out, want), (x["state"], S))]
    print(dt, width, "relative error", rel)
    assert rel[0] <= {F32: 1e-6, BF16: 4e-3, F16: 4e-4}[dt] and rel[1] <= 1e-6


def test_strided_rows_and_views(o1):
    """q, k, v and out as slices of wider rows, as a fused projection leaves them."""
    G, hpg, d, dv, rows = 2, 2, 64, 48, 210
    x = make(G, hpg, d, dv, rows, 1, BF16, 11)
    nq, nk, nv = G * hpg * d, G * d, G * dv
    wide = torch.full((rows, nq + nk + nv + 24), float("nan"), dtype=BF16, device="cuda")
    for n, o, h, w in (("q", 0, G * hpg, d), ("k", nq, G, d), ("v", nq + nk, G, dv)):
        wide[:, o:o + h * w] = x[n].flatten(1)
        x[n] = wide[:, o:o + h * w].unflatten(1, (h, w))
    outw = torch.full((rows, G * hpg * dv + 8), float("nan"), dtype=BF16, device="cuda")
    out = outw[:, 8:].unflatten(1, (G * hpg, dv))
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=BF16), x["state"].clone()
    chunk(o1, x, geom, [(0, rows, 0)], out)
    torch.cuda.synchronize()
    check(o1, x, s0, [(0, rows, 0)], out, geom.scale, "strided")
    assert torch.isnan(outw[:, :8]).all()


def test_passes_of_a_small_scratch(o1):
    """The smallest scratch: the same rows in many passes."""
    G, hpg, d, dv, lens = 1, 2, 64, 64, [700, 90, 1, 300]
    x = make(G, hpg, d, dv, sum(lens), 4, F32, 13)
    geom, s0 = o1.lin_geom(G, hpg, d, dv), x["state"].clone()
    seqs = [(sum(lens[:i]), n, 3 - i) for i, n in enumerate(lens)]
    out = torch.full((sum(lens), 2, dv), float("nan"), device="cuda")
    chunk(o1, x, geom, seqs, out, scratch_rows=1)
    torch.cuda.synchronize()
    check(o1, x, s0, seqs, out, geom.scale, "small scratch")


def test_more_sequences_than_a_launch_takes(o1):
    lens = [(7 * i) % 40 for i in range(300)] + [200, 150]
    x = make(1, 1, 16, 16, sum(lens), len(lens), F32, 17)
    geom, s0 = o1.lin_geom(1, 1, 16, 16), x["state"].clone()
    seqs = [(sum(lens[:i]), n, len(lens) - 1 - i) for i, n in enumerate(lens)]
    seqs = seqs[::-1]
    out = torch.full((sum(lens), 1, 16), float("nan"), device="cuda")
    chunk(o1, x, geom, seqs, out)
    torch.cuda.synchronize()
    check(o1, x, s0, seqs, out, geom.scale, "many sequences")


def test_split_calls_and_tokens_carry_on(o1):
    """A prompt in two calls, then rows one at a time: one sequence."""
    G, hpg, d, dv, rows = 2, 2, 128, 128, 410
    x = make(G, hpg, d, dv, rows, 3, F32, 19)
    geom, s0 = o1.lin_geom(G, hpg, d, dv), x["state"].clone()
    out = torch.full((rows, 4, dv), float("nan"), device="cuda")
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    chunk(o1, x, geom, [(0, 250, 2)], out)
    chunk(o1, x, geom, [(250, 150, 2)], out)
    for r in range(400, rows):
        o1.check(o1.o1_lin_token_attend(x["state"], geom, x["q"][r:r + 1], x["k"][r:r + 1], x["v"][r:r + 1], x["g"], slots,
                                        out[r:r + 1]))
    torch.cuda.synchronize()
    check(o1, x, s0, [(0, rows, 2)], out, geom.scale, "carried on")


TOKENS = [
    (2, 4, 256, 256, 1, 1, F32), (4, 4, 128, 128, 40, 48, BF16), (1, 1, 8, 8, 3, 3, F32), (3, 2, 72, 40, 17, 20, F16),
    (1, 3, 256, 8, 5, 9, BF16), (2, 1, 64, 200, 300, 310, F32), (1, 16, 16, 16, 2, 2, F16),
]


@pytest.mark.parametrize("case", range(len(TOKENS)))
def test_token(o1, case):
    G, hpg, d, dv, rows, slots, dt = TOKENS[case]
    x = make(G, hpg, d, dv, rows, slots, dt, 200 + case, [-0.3, 0.0, -1e-3, float("-inf")] if case % 2 else None)
    gen = torch.Generator().manual_seed(case)
    idx = torch.randperm(slots, generator=gen)[:rows].to(torch.int32)
    if rows > 4:   # padding, a slot past the end, a slot named twice
        idx[1], idx[2], idx[rows - 1] = -1, slots, idx[0]
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=dt), x["state"].clone()
    out = torch.full((rows, G * hpg, dv), float("nan"), dtype=dt, device="cuda")
    o1.check(o1.o1_lin_token_attend(x["state"], geom, x["q"], x["k"], x["v"], x["g"], idx.cuda(), out))
    torch.cuda.synchronize()
    seqs = [(r, 1, int(i)) for r, i in enumerate(idx.tolist()) if 0 <= i < slots and i not in idx[:r].tolist()]
    check(o1, x, s0, seqs, out, geom.scale, f"token {case}")


def test_token_without_slots_and_strided(o1):
    x = make(2, 2, 64, 64, 5, 6, BF16, 31)
    wide = torch.zeros(5, 4 * 64 + 16, dtype=BF16, device="cuda")
    wide[:, 16:] = x["q"].flatten(1)
    x["q"] = wide[:, 16:].unflatten(1, (4, 64))
    geom, s0 = o1.lin_geom(2, 2, 64, 64, dtype=BF16), x["state"].clone()
    out = torch.full((5, 4, 64), float("nan"), dtype=BF16, device="cuda")
    o1.check(o1.o1_lin_token_attend(x["state"], geom, x["q"], x["k"], x["v"], x["g"], None, out))
    check(o1, x, s0, [(r, 1, r) for r in range(5)], out, geom.scale, "no slots")


def test_binding_refuses_wrong_tensors(o1):
    x = make(2, 2, 64, 64, 5, 6, F32, 31)
    geom = o1.lin_geom(2, 2, 64, 64)
    out = torch.empty(5, 4, 64, device="cuda")
    call = lambda **kw: o1.o1_lin_token_attend(*[{**x, "geom": geom, "slots": None, "out": out, **kw}[n] for n in
                                                 ("state", "geom", "q", "k", "v", "g", "slots", "out")])
    assert call() == o1.O1_OK
    for bad, err in ((dict(q=x["q"].cpu()), TypeError), (dict(q=x["q"].half()), TypeError), (dict(v=x["v"][:4]), ValueError),
                     (dict(k=x["k"].transpose(1, 2)), ValueError), (dict(state=x["state"][:, :3]), ValueError),
                     (dict(slots=torch.zeros(5, device="cuda", dtype=torch.int64)), TypeError),
                     (dict(slots=torch.zeros(4, device="cuda", dtype=torch.int32)), ValueError),
                     (dict(g=x["g"][:3]), ValueError), (dict(state=x["state"].double()), TypeError)):
        with pytest.raises(err):
            call(**bad)
    assert call(q=x["q"][:1].expand(5, 4, 64)) == o1.O1_ERR_ARG   # rows on top of one another


def test_captured_token_step_replays_on_other_slots(o1):
    rows, slots = 6, 12
    x = make(2, 2, 64, 64, rows, slots, BF16, 37)
    geom, s0 = o1.lin_geom(2, 2, 64, 64, dtype=BF16), x["state"].clone()
    idx = torch.arange(rows, dtype=torch.int32, device="cuda")
    out = torch.full((rows, 4, 64), float("nan"), dtype=BF16, device="cuda")
    step = lambda: o1.check(o1.o1_lin_token_attend(x["state"], geom, x["q"], x["k"], x["v"], x["g"], idx, out))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x["state"].copy_(s0)
    idx.copy_(torch.tensor([11, -1, 3, 3, 0, 7], dtype=torch.int32))
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check(o1, x, s0, [(0, 1, 11), (2, 1, 3), (4, 1, 0), (5, 1, 7)], out, geom.scale, "replay")


def test_captured_chunk_replays(o1):
    x = make(2, 2, 64, 64, 400, 2, F32, 41)
    geom, s0 = o1.lin_geom(2, 2, 64, 64), x["state"].clone()
    seqs = [(0, 300, 1), (300, 100, 0)]
    out = torch.full((400, 4, 64), float("nan"), device="cuda")
    scratch = torch.empty(o1.o1_lin_scratch_bytes(geom, 400, 2), dtype=torch.uint8, device="cuda")
    run = lambda: o1.check(o1.o1_lin_chunk_attend(x["state"], geom, scratch, x["q"], x["k"], x["v"], x["g"], seqs, out))
    run()
    torch.cuda.synchronize()
    first, after = out.clone(), x["state"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    x["state"].copy_(s0)
    out.fill_(float("nan"))
    scratch.fill_(255)       # whatever the scratch holds
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(x["state"], after)
    check(o1, x, s0, seqs, out, geom.scale, "replayed chunk")


def test_other_stream_and_repeatable(o1):
    x = make(1, 4, 128, 128, 300, 1, BF16, 43)
    geom, s0 = o1.lin_geom(1, 4, 128, 128, dtype=BF16), x["state"].clone()
    st = torch.cuda.Stream()
    got = []
    for stream in (None, st, st):
        x["state"].copy_(s0)
        out = torch.full((300, 4, 128), float("nan"), dtype=BF16, device="cuda")
        torch.cuda.synchronize()
        scratch = chunk(o1, x, geom, [(0, 300, 0)], out, stream=stream)
        torch.cuda.synchronize()
        got.append((out, x["state"].clone()))
        del scratch
    for o, s in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(s, got[0][1])


def test_state_past_32_bit_offsets(o1):
    """The last slot of a state of more than 2^31 values."""
    G, hpg, d, dv = 1, 16, 256, 256
    geom = o1.lin_geom(G, hpg, d, dv)
    slots = 2 ** 31 // (16 * 65536) + 2
    small = make(G, hpg, d, dv, 130, 1, F32, 47)
    big = torch.empty(slots, 16, d, dv, device="cuda")
    big[-1] = small["state"][0]
    out = torch.full((130, 16, dv), float("nan"), device="cuda")
    x = {**small, "state": big}
    chunk(o1, x, geom, [(0, 129, slots - 1)], out)
    o1.check(o1.o1_lin_token_attend(big, geom, x["q"][129:], x["k"][129:], x["v"][129:], x["g"],
                                    torch.tensor([slots - 1], dtype=torch.int32, device="cuda"), out[129:]))
    torch.cuda.synchronize()
    y = {**small, "state": big[-1:].clone()}
    del big
    check(o1, y, small["state"], [(0, 130, 0)], out, geom.scale, "large state")


def test_prep_prompt_and_tokens_together(o1):
    """As used: heads normalised and rotated, a prompt, then single rows."""
    G, hpg, d, dv, rows = 2, 2, 128, 64, 203
    x = make(G, hpg, d, dv, rows, 1, F32, 53)
    gp = o1.prep_geom(G * hpg, G, d)
    inv = (1e6 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    wq, wk = 1 + 0.1 * torch.randn(d).cuda(), 1 + 0.1 * torch.randn(d).cuda()
    geom, s0 = o1.lin_geom(G, hpg, d, dv), x["state"].clone()
    out = torch.full((rows, G * hpg, dv), float("nan"), device="cuda")
    pq, pk = torch.empty_like(x["q"]), torch.empty_like(x["k"])
    scratch = torch.empty(o1.o1_lin_scratch_bytes(geom, rows), dtype=torch.uint8, device="cuda")
    for r0, r1 in [(0, 200)] + [(r, r + 1) for r in range(200, rows)]:
        s = slice(r0, r1)
        o1.check(o1.o1_head_prep(gp, x["q"][s], x["k"][s], wq, wk, inv, pq[s], pk[s], pos0=r0))
        if r1 - r0 > 1:
            o1.check(o1.o1_lin_chunk_attend(x["state"], geom, scratch, pq[s], pk[s], x["v"][s], x["g"], [(0, r1 - r0, 0)],
                                            out[s]))
        else:
            o1.check(o1.o1_lin_token_attend(x["state"], geom, pq[s], pk[s], x["v"][s], x["g"], None, out[s]))
    torch.cuda.synchronize()
    pos = torch.arange(rows)
    for src, w, got in ((x["q"], wq, pq), (x["k"], wk, pk)):
        z, mag = ref.prep(src, w, inv, pos, d, "rms", 1e-6)
        ref.assert_within(got, z, ref.prep_bound(z, mag, d, F32), "prep")
    check(o1, {**x, "q": pq, "k": pk}, s0, [(0, rows, 0)], out, geom.scale, "together")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_expired_waits_raise_the_flag(o1, dt):
    """Waits cut to a clock cycle run out: the call ends, the flag is raised, what its
    blocks would have written is NaN, and with the limit restored the next
    call is right again."""
    x = make(2, 2, 128, 128, 600, 1, dt, 59)
    geom, s0 = o1.lin_geom(2, 2, 128, 128, dtype=dt), x["state"].clone()
    assert o1.o1_lin_flags() == 0
    out = torch.zeros(600, 4, 128, dtype=dt, device="cuda")
    o1.o1_set_wait_limit(1)
    try:
        chunk(o1, x, geom, [(0, 600, 0)], out)
        torch.cuda.synchronize()
    finally:
        o1.o1_set_wait_limit(0)
    assert o1.o1_lin_flags(clear=True) == o1.O1_FLAG_WAIT_EXPIRED
    assert o1.o1_lin_flags() == 0
    assert torch.isnan(out).any()
    x["state"].copy_(s0)
    out.fill_(float("nan"))
    chunk(o1, x, geom, [(0, 600, 0)], out)
    torch.cuda.synchronize()
    check(o1, x, s0, [(0, 600, 0)], out, geom.scale, "after expiry")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_a_sequence_of_nans_spoils_no_neighbour(o1, dt):
    """Three sequences end to end, the middle one NaN and infinities throughout."""
    lens = [150, 70, 140]
    x = make(2, 2, 64, 72, sum(lens), 3, dt, 61)
    for n, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan"))):
        x[n][lens[0]:lens[0] + lens[1]] = bad
    geom, s0 = o1.lin_geom(2, 2, 64, 72, dtype=dt), x["state"].clone()
    seqs = [(sum(lens[:i]), n, i) for i, n in enumerate(lens)]
    out = torch.zeros(sum(lens), 4, 72, dtype=dt, device="cuda")
    chunk(o1, x, geom, seqs, out)
    torch.cuda.synchronize()
    assert torch.isnan(out[lens[0]:lens[0] + lens[1]]).all()
    keep = [seqs[0], seqs[2]]
    y = {**x, "state": torch.stack([x["state"][0], s0[1], x["state"][2]])}
    for r0, n, _ in [seqs[1]]:
        out[r0:r0 + n] = float("nan")
    check(o1, {**y, **{n: torch.nan_to_num(x[n], 0, 0, 0) for n in "qkv"}}, s0, keep, out, geom.scale, "neighbours")


def test_rows_past_32_bit_offsets(o1):
    """A row stride of 2^27 values: rows past 2^31 values from the first."""
    rows, d = 40, 64
    x = make(1, 1, d, d, rows, 1, BF16, 67)
    geom, s0 = o1.lin_geom(1, 1, d, d, dtype=BF16), x["state"].clone()
    far = torch.empty(rows << 27, dtype=BF16, device="cuda")
    q = far.as_strided((rows, 1, d), (1 << 27, d, 1))
    k = far[4096:].as_strided((rows, 1, d), (1 << 27, d, 1))
    out = far[8192:].as_strided((rows, 1, d), (1 << 27, d, 1))
    q.copy_(x["q"])
    k.copy_(x["k"])
    chunk(o1, {**x, "q": q, "k": k}, geom, [(0, rows, 0)], out)
    torch.cuda.synchronize()
    got = out.clone()
    del far, q, k, out
    check(o1, x, s0, [(0, rows, 0)], got, geom.scale, "far rows")


def test_two_streams_with_a_scratch_each(o1):
    xs = [make(2, 2, 128, 128, 900, 1, F32, 71 + i) for i in range(2)]
    geom = o1.lin_geom(2, 2, 128, 128)
    s0 = [x["state"].clone() for x in xs]
    outs = [torch.full((900, 4, 128), float("nan"), device="cuda") for _ in xs]
    scr = [torch.empty(o1.o1_lin_scratch_bytes(geom, 900), dtype=torch.uint8, device="cuda") for _ in xs]
    st = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        o1.check(o1.o1_lin_chunk_attend(x["state"], geom, scr[i], x["q"], x["k"], x["v"], x["g"], [(0, 900, 0)], outs[i],
                                        stream=st[i]))
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        check(o1, x, s0[i], [(0, 900, 0)], outs[i], geom.scale, f"stream {i}")


def test_a_scratch_of_one_step_serves_every_type(o1):
    """The least scratch holds one state and a few rows: steps of 16 rows."""
    for dt in (F32, BF16, F16):
        x = make(1, 2, 136, 72, 210, 1, dt, 73)
        geom, s0 = o1.lin_geom(1, 2, 136, 72, dtype=dt), x["state"].clone()
        out = torch.full((210, 2, 72), float("nan"), dtype=dt, device="cuda")
        chunk(o1, x, geom, [(0, 210, 0)], out, scratch_rows=1)
        torch.cuda.synchronize()
        check(o1, x, s0, [(0, 210, 0)], out, geom.scale, f"least scratch {dt}")


@pytest.mark.parametrize("limit", [1, 2000])
@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_expired_waits_spoil_values_with_nan_only(o1, dt, limit):
    """Waits that run out at once, or some of them: every value is NaN or right,
    and a NaN that is not raised by the flag does not occur."""
    G, hpg, d, dv = 4, 2, 72, 136
    lens = [700, 129, 256, 64, 513]
    x = make(G, hpg, d, dv, sum(lens), len(lens), dt, 101)
    seqs = [(sum(lens[:i]), n, i) for i, n in enumerate(lens)]
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=dt), x["state"].clone()
    want, Ao, S, As = ref.linear(x["q"], x["k"], x["v"], x["g"], s0, seqs, geom.scale)
    bo, bs = ref.linear_bounds(want, Ao, As, seqs, dt)
    for _ in range(3):
        x["state"].copy_(s0)
        out = torch.zeros(sum(lens), G * hpg, dv, dtype=dt, device="cuda")
        o1.o1_set_wait_limit(limit)
        try:
            chunk(o1, x, geom, seqs, out)
            torch.cuda.synchronize()
        finally:
            o1.o1_set_wait_limit(0)
        expired = o1.o1_lin_flags(clear=True) == o1.O1_FLAG_WAIT_EXPIRED
        assert expired or limit > 1
        for got, w, b in ((out, want, bo), (x["state"], S, bs)):
            got = got.cpu().double()
            bad = torch.isnan(got)
            assert expired or not bad.any()
            assert ((got - w).abs() <= b)[~bad].all()


def test_more_rows_than_a_call_counts(o1):
    """A row count past 32 bits is refused, not taken modulo 2^32."""
    geom = o1.lin_geom(1, 1, 8, 8)
    t = torch.zeros(1, 1, 8, device="cuda").expand(2 ** 32 + 1, 1, 8)
    state, g = torch.zeros(1, 1, 8, 8, device="cuda"), torch.zeros(1, device="cuda")
    with pytest.raises(ValueError):
        o1.o1_lin_token_attend(state, geom, t, t, t, g, None, t)
    with pytest.raises(ValueError):
        o1.o1_lin_chunk_attend(state, geom, torch.empty(4096, dtype=torch.uint8, device="cuda"), t, t, t, g, [(0, 1, 0)], t)


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("before", ["kernel", "copy", "join", "prep"])
def test_captured_behind_other_work(o1, dt, before):
    """A captured prompt whose queries come from a foreign kernel, a copy, another
    stream, or the head prep just before it: every replay takes the new ones."""
    G, hpg, d, dv, rows = 2, 2, 64, 64, 420
    x = make(G, hpg, d, dv, rows, 2, dt, 83)
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=dt), x["state"].clone()
    seqs = o1.lin_seqs([(0, 300, 1), (300, 120, 0)])
    out = torch.full((rows, G * hpg, dv), float("nan"), dtype=dt, device="cuda")
    scratch = torch.empty(o1.o1_lin_scratch_bytes(geom, rows, 2), dtype=torch.uint8, device="cuda")
    src, side = torch.empty_like(x["q"]), torch.cuda.Stream()
    copy_of = lambda: x["q"].copy_(src)
    gp = o1.prep_geom(G * hpg, 0, d, rot=0, norm="none", in_dtype=dt)

    def run():
        here = torch.cuda.current_stream()
        if before == "kernel":
            torch.mul(src, 1.0, out=x["q"])
        elif before == "copy":
            copy_of()
        elif before == "prep":
            o1.check(o1.o1_head_prep(gp, src, None, None, None, None, x["q"], None))
        else:
            side.wait_stream(here)
            with torch.cuda.stream(side):
                copy_of()
            torch.add(x["v"], 0.0, out=x["v"])
            here.wait_stream(side)
        o1.check(o1.o1_lin_chunk_attend(x["state"], geom, scratch, x["q"], x["k"], x["v"], x["g"], seqs, out))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (1, 2):
        src.copy_(torch.randn(src.shape, generator=torch.Generator().manual_seed(seed)).to(dt))
        x["q"].fill_(float("nan"))
        out.fill_(float("nan"))
        x["state"].copy_(s0)
        graph.replay()
        torch.cuda.synchronize()
        check(o1, {**x, "q": src}, s0, [(0, 300, 1), (300, 120, 0)], out, geom.scale, f"behind a {before}")


def launches(run):
    """How many nodes a call leaves in a captured graph: its launches."""
    import ctypes
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        run()
    n = ctypes.c_size_t(0)
    cudart = ctypes.CDLL(next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart.so" in line))
    assert cudart.cudaGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_short_sequences_of_a_small_scratch(o1, dt):
    """With a scratch of one state each sequence sent to the tiles is a pass of
    its own: 32 short ones go by rows, in one launch."""
    G, hpg, d, n, r = 2, 2, 128, 32, 24
    x = make(G, hpg, d, d, n * r, n, dt, 97)
    geom, s0 = o1.lin_geom(G, hpg, d, d, dtype=dt), x["state"].clone()
    seqs = [(r * i, r, i) for i in range(n)]
    out = torch.full((n * r, G * hpg, d), float("nan"), dtype=dt, device="cuda")
    scratch = torch.empty(o1.o1_lin_scratch_bytes(geom, 1), dtype=torch.uint8, device="cuda")
    call = lambda: o1.check(o1.o1_lin_chunk_attend(x["state"], geom, scratch, x["q"], x["k"], x["v"], x["g"], seqs, out))
    call()
    torch.cuda.synchronize()
    assert launches(call) == 1
    x["state"].copy_(s0)
    chunk(o1, x, geom, seqs, out, scratch_rows=1)
    torch.cuda.synchronize()
    check(o1, x, s0, seqs, out, geom.scale, "small scratch by rows")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
def test_passes_of_long_segments(o1, dt):
    """More tiles than SMs (segments of 256 rows) in many passes: the least
    scratch (steps of 16 rows, of a segment for bf16), one that takes 128 rows
    but not a segment's panels, one of several segments. Sequences are cut at
    each and carry on from their slots."""
    G, hpg, d, dv = 4, 2, 72, 136
    lens = [700, 129, 130, 256, 64, 255, 257, 300, 128, 513, 49, 1025, 384, 100]
    rows = sum(lens)
    x = make(G, hpg, d, dv, rows, len(lens), dt, 89)
    seqs = [(sum(lens[:i]), n, len(lens) - 1 - i) for i, n in enumerate(lens)]
    geom, s0 = o1.lin_geom(G, hpg, d, dv, dtype=dt), x["state"].clone()
    want, Ao, S, As = ref.linear(x["q"], x["k"], x["v"], x["g"], s0, seqs, geom.scale)
    bo, bs = ref.linear_bounds(want, Ao, As, seqs, dt)
    for scratch_rows in (1, 128, 512, 900):
        x["state"].copy_(s0)
        out = torch.full((rows, G * hpg, dv), float("nan"), dtype=dt, device="cuda")
        chunk(o1, x, geom, seqs, out, scratch_rows=scratch_rows)
        torch.cuda.synchronize()
        ref.assert_within(out, want, bo, f"scratch of {scratch_rows} rows, out")
        ref.assert_within(x["state"], S, bs, f"scratch of {scratch_rows} rows, state")


def test_flags_of_two_streams(o1):
    """A flag raised on one stream stays until it is read as raised, whichever
    stream reads, with or without a reset; reads that find none drop none."""
    x = make(2, 2, 128, 128, 600, 1, BF16, 103)
    geom = o1.lin_geom(2, 2, 128, 128, dtype=BF16)
    out, st = torch.zeros(600, 4, 128, dtype=BF16, device="cuda"), torch.cuda.Stream()
    assert o1.o1_lin_flags(clear=True) == 0
    torch.cuda.synchronize()
    o1.o1_set_wait_limit(1)
    try:
        keep = chunk(o1, x, geom, [(0, 600, 0)], out, stream=st)
        seen = [o1.o1_lin_flags(clear=True) for _ in range(50)]   # beside the running call
    finally:
        o1.o1_set_wait_limit(0)
    torch.cuda.synchronize()
    del keep
    seen += [o1.o1_lin_flags(), o1.o1_lin_flags(clear=True, stream=st)]
    assert o1.O1_FLAG_WAIT_EXPIRED in seen and set(seen) <= {0, o1.O1_FLAG_WAIT_EXPIRED}
    o1.o1_lin_flags(clear=True)
    assert o1.o1_lin_flags() == 0
