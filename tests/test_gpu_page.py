"""The paged cache on the GPU against 64-bit references: what a write holds and
what it leaves alone, reading back, attention of chunks and of single rows over
all types, head layouts, widths, pages, windows, lengths from one to thousands;
garbage where nothing is attended, absent pages, padding, strides, capture and
replay, streams, and the operators run together as a model runs them."""
import pytest
import torch

import pg_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16, F16, E4 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(F32, BF16), (F32, E4), (BF16, BF16), (BF16, E4), (F16, F16), (F16, E4)]
NAN = float("nan")


@pytest.fixture(scope="module")
def o1():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sliding_window_landmark_gb300 import build
    build.build()
    from sliding_window_landmark_gb300 import o1 as mod
    return mod


class Cache:
    """A cache of random values over a table of its own order. `ends`: positions
    held of each slot; what lies past them holds NaN (and bytes of 255), and the
    table's entries past them name no page."""

    def __init__(self, o1, g, ends, seed, spare=2, fill=True):
        gen = torch.Generator().manual_seed(seed)
        self.g, self.ct = g, o1._CACHE_TYPES[g.cache_dtype]
        used = [-(-n // g.page) for n in ends]
        self.n = sum(used) + spare
        ids = torch.randperm(self.n, generator=gen).to(torch.int32)
        table = torch.full((len(ends), max(used + [1]) + 1), -1, dtype=torch.int32)
        table[:, -1] = 2 ** 31 - 1
        at = 0
        for s, n in enumerate(used):
            table[s, :n] = ids[at:at + n]
            at += n
        self.table = table.cuda()
        self.k, self.v, self.ke, self.ve = self._pool(g.d, gen, fill), self._pool(g.dv, gen, fill), None, None
        if self.ct is E4:
            self.ke, self.ve = (torch.randint(116, 122, (self.n, g.groups, g.page), generator=gen).to(torch.uint8).cuda() for _ in "kv")
        if fill:
            held = torch.zeros(self.n, g.page, dtype=torch.bool)
            for s, n in enumerate(ends):
                p = torch.arange(n)
                held[table[s, p // g.page].long(), p % g.page] = True
            gone = (~held).cuda()[:, None].expand(-1, g.groups, -1)
            for x, e in ((self.k, self.ke), (self.v, self.ve)):
                if e is None:
                    x[gone] = NAN
                else:
                    x.view(torch.uint8)[gone] = 0x7f
                    e[gone] = 255
        self.c = o1.pg_cache(g, self.k, self.v, self.table, self.ke, self.ve)

    def _pool(self, w, gen, fill):
        x = torch.randn(self.n, self.g.groups, self.g.page, w, generator=gen) if fill else torch.zeros(self.n, self.g.groups, self.g.page, w)
        return (x * 90).clamp(-448, 448).to(E4).cuda() if self.ct is E4 else x.to(self.ct).cuda()

    def held(self):
        return ref.held(self.k, self.ke), ref.held(self.v, self.ve)

    def raw(self):
        return [x.view(torch.uint8).clone() for x in (self.k, self.v, self.ke, self.ve) if x is not None]


def randn(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def attend(o1, cache, q, seqs, out, stream=None, token=None):
    g = cache.g
    scratch = torch.empty(o1.o1_pg_scratch_bytes(g, q.shape[0]), dtype=torch.uint8, device="cuda")
    scratch.fill_(0xff)   # NaN and counts of -1, should anything be read before it is written
    if token:
        o1.check(o1.o1_pg_token_attend(g, cache.c, scratch, q, token[0], token[1], out, stream=stream), "token")
    else:
        o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, q, seqs, out, stream=stream), "chunk")
    return scratch


def check(o1, cache, q, seqs, out, what):
    g = cache.g
    k, v = cache.held()
    dt = q.dtype
    terms, rho, f16 = ref.precision(dt, cache.ct)
    want, bound = ref.attend(q, k, v, cache.table, g.page, cache.n, seqs, g.scale, g.window, dt, terms, rho, f16, cache.ve)
    live = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for r0, n, _, _ in seqs:
        live[r0:r0 + n] = True
    ref.assert_within(out[live], want[live].cpu(), bound[live].cpu(), what)
    assert torch.isnan(out[~live]).all(), what + ": rows of no sequence were written"


def spread(lens, pasts, slots):
    """Sequences with a row of none before and two after; slots in an order of their own."""
    seqs, r = [], 1
    for i, (n, p) in enumerate(zip(lens, pasts)):
        seqs.append((r, n, (2 * i + 1) % slots if slots % 2 else (i + 1) % slots, p))
        r += n
    ends = [0] * slots
    for _, n, s, p in seqs:
        ends[s] = n + p
    return seqs, ends, r + 2


# ------------------------------------------------------------------ the cache

# G, d, dv, page, lengths, pasts
COPIES = [
    (1, 8, 8, 16, [1], [0]),
    (2, 256, 256, 64, [1, 0, 2], [8191, 3, 15]),
    (3, 72, 40, 32, [1000, 77], [3, 130]),
    (4, 128, 128, 16, [70, 1, 0, 257, 33, 128, 5], [0, 15, 2, 16, 17, 31, 1000]),
    (1, 16, 256, 256, [300], [255]),
    (5, 64, 96, 128, [129, 3], [0, 127]),
    (2, 32, 32, 16, [1] * 300, list(range(300))),
]


def unit(ct, w):
    return -(-w // 16) * 16 if ct is E4 else w


@pytest.mark.parametrize("case", range(len(COPIES)))
@pytest.mark.parametrize("dt,ct", TYPES)
def test_write_and_read(o1, dt, ct, case):
    G, d, dv, page, lens, pasts = COPIES[case]
    d, dv = unit(ct, d), unit(ct, dv)
    seqs, ends, rows = spread(lens, pasts, len(lens) + 1)
    g = o1.pg_geom(G, 2, d, dv, page, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, ends, case)
    gen = torch.Generator().manual_seed(50 + case)
    # fused rows, a stride of more than a row; heads of very different sizes, zeros, infinities and NaN
    fused = randn(gen, rows, G * (d + dv) + 8) * torch.exp2(6 * randn(gen, rows, 1))
    fused[2 % rows] = 0.0
    fused = fused.clamp(-6e4, 6e4).to(dt)
    k, v = fused[:, :G * d].unflatten(1, (G, d)), fused[:, G * d:G * (d + dv)].unflatten(1, (G, dv))
    if rows > 8:
        k[4, 0, 3], v[5, G - 1, 7], k[6] = float("inf"), NAN, -float("inf")
    k[0], v[0], k[-2:], v[-2:] = NAN, NAN, NAN, NAN    # rows of no sequence
    before = cache.raw()
    o1.check(o1.o1_pg_write(g, cache.c, k, v, seqs), "write")
    touched = torch.zeros(cache.n, page, dtype=torch.bool, device="cuda")
    back_k, back_v = torch.full((rows, G, d), NAN, dtype=dt, device="cuda"), torch.full((rows, G, dv), NAN, dtype=dt, device="cuda")
    back_k[0], back_v[-1] = 7.0, 9.0
    o1.check(o1.o1_pg_read(g, cache.c, seqs, back_k, back_v), "read")
    for r0, n, slot, p in seqs:
        if not n:
            continue
        ids, at = ref.places(cache.table, page, slot, p, p + n)
        touched[ids, at] = True
        for x, pool, exp, back in ((k, cache.k, cache.ke, back_k), (v, cache.v, cache.ve, back_v)):
            x = x[r0:r0 + n]
            if ct is E4:
                want, byte = ref.quantise(x)
                assert torch.equal(exp[ids, :, at], byte)
                got = ref.held(pool, exp)[ids, :, at]
            else:
                want, got = x.to(ct).double(), pool[ids, :, at].double()
            torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)
            torch.testing.assert_close(back[r0:r0 + n].double(), want.to(dt).double(), rtol=0, atol=0, equal_nan=True)
    for old, new in zip(before, cache.raw()):
        keep = (~touched)[:, None].expand(-1, G, -1)
        assert torch.equal(old[keep], new[keep]), "a position of no row was written"
    assert (back_k[0] == 7).all() and (back_v[-1] == 9).all() and torch.isnan(back_k[-2:]).all(), "rows of no sequence were written"


@pytest.mark.parametrize("ct", [BF16, E4])
def test_absent_pages_are_left_out(o1, ct):
    G, d, page = 2, 64, 16
    g = o1.pg_geom(G, 2, d, d, page, dtype=F32, cache_dtype=ct)
    cache = Cache(o1, g, [100, 40], 3)
    cache.table[0, 1], cache.table[0, 4] = -1, cache.n    # positions 16 .. 31 and 64 .. 79
    gen = torch.Generator().manual_seed(1)
    k, v = randn(gen, 100, G, d), randn(gen, 100, G, d)
    before = cache.raw()
    o1.check(o1.o1_pg_write(g, cache.c, k, v, [(0, 100, 0, 0)]), "write")
    back = torch.full((100, G, d), 5.0, device="cuda"), torch.full((100, G, d), 5.0, device="cuda")
    o1.check(o1.o1_pg_read(g, cache.c, [(0, 100, 0, 0)], *back), "read")
    gone = torch.tensor([p // 16 in (1, 4) for p in range(100)], device="cuda")
    for x, b in zip((k, v), back):
        assert (b[gone] == 5).all()
        assert torch.equal(b[~gone], (ref.quantise(x)[0] if ct is E4 else x.to(ct)).float()[~gone])
    ids = torch.ones(cache.n, dtype=torch.bool, device="cuda")
    ids[cache.table[0, [0, 2, 3, 5, 6]].long()] = False
    assert all(torch.equal(a[ids], b[ids]) for a, b in zip(before, cache.raw()))
    # attended: without them; a row whose window holds only absent ones is 0
    q = randn(gen, 100, 4, d)
    for window in (0, 10):
        g.window = window
        out = torch.full((100, 4, d), NAN, device="cuda")
        attend(o1, cache, q, [(0, 100, 0, 0)], out)
        check(o1, cache, q, [(0, 100, 0, 0)], out, f"absent pages, window {window}")
        assert not window or (out[26:32] == 0).all()
        pos, slots = torch.arange(100, device="cuda"), torch.zeros(100, dtype=torch.int32, device="cuda")
        out = torch.full((100, 4, d), NAN, device="cuda")
        attend(o1, cache, q, None, out, token=(slots, pos))
        check(o1, cache, q, [(r, 1, 0, r) for r in range(100)], out, f"absent pages, rows, window {window}")


@pytest.mark.parametrize("dt,ct", TYPES)
def test_token_write(o1, dt, ct):
    G, d, dv, page = 3, 80, 48, 32
    g = o1.pg_geom(G, 1, d, dv, page, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, [70, 33, 200, 1, 64], 5)
    gen = torch.Generator().manual_seed(2)
    # row: slot, position; padding by slot and by position, an absent page, a place named three times
    rows = [(2, 199), (0, 0), (-1, 3), (5, 3), (0, 69), (1, -1), (1, 10 ** 12), (2, 199), (4, 32), (0, 1), (2, 199), (1, 64), (3, 0)]
    slots = torch.tensor([s for s, _ in rows], dtype=torch.int32, device="cuda")
    pos = torch.tensor([p for _, p in rows], dtype=torch.int64, device="cuda")
    k, v = randn(gen, len(rows), G, d, dtype=dt), randn(gen, len(rows), G, dv, dtype=dt)
    before = cache.raw()
    o1.check(o1.o1_pg_token_write(g, cache.c, k, v, slots, pos), "write")
    touched = torch.zeros(cache.n, page, dtype=torch.bool, device="cuda")
    for r in (0, 1, 4, 8, 9, 12):
        ids, at = ref.places(cache.table, page, rows[r][0], rows[r][1], rows[r][1] + 1)
        touched[ids, at] = True
        for x, pool, exp in ((k, cache.k, cache.ke), (v, cache.v, cache.ve)):
            if ct is E4:
                want, byte = ref.quantise(x[r:r + 1])
                assert torch.equal(exp[ids, :, at], byte) and torch.equal(ref.held(pool, exp)[ids, :, at], want)
            else:
                assert torch.equal(pool[ids, :, at], x[r:r + 1].to(ct))
    for old, new in zip(before, cache.raw()):
        keep = (~touched)[:, None].expand(-1, G, -1)
        assert torch.equal(old[keep], new[keep])
    # no slots: row r is slot r's
    o1.check(o1.o1_pg_token_write(g, cache.c, k[:5], v[:5], None, torch.zeros(5, dtype=torch.int64, device="cuda")), "write")
    for r in range(5):
        ids, at = ref.places(cache.table, page, r, 0, 1)
        want = ref.quantise(k[r:r + 1])[0] if ct is E4 else k[r:r + 1].to(ct).double()
        assert torch.equal(ref.held(cache.k, cache.ke)[ids, :, at], want)


# -------------------------------------------------------------- the attention

# G, hpg, d, dv, page, window, lengths, pasts
CHUNKS = [
    (1, 1, 64, 64, 16, 0, [1], [0]),
    (1, 2, 64, 64, 16, 0, [2], [0]),
    (2, 1, 64, 64, 64, 0, [65], [0]),
    (2, 4, 128, 128, 64, 0, [130], [0]),
    (2, 4, 256, 256, 64, 0, [70], [500]),
    (1, 3, 8, 8, 16, 0, [50], [13]),
    (1, 16, 32, 32, 128, 0, [40], [1000]),
    (3, 3, 72, 40, 32, 0, [150, 77], [0, 1001]),
    (2, 5, 200, 136, 16, 0, [90, 140], [7, 250]),
    (1, 4, 16, 256, 32, 0, [70], [60]),
    (1, 4, 256, 16, 32, 0, [70], [60]),
    (4, 4, 128, 128, 16, 0, [70, 1, 0, 257, 33, 128, 5], [0, 700, 9, 128, 127, 2000, 64]),
    (2, 2, 128, 128, 64, 1, [100], [30]),
    (2, 2, 64, 128, 16, 50, [300, 20], [0, 333]),
    (1, 4, 128, 64, 256, 200, [513], [300]),
    (2, 4, 128, 128, 64, 129, [1000], [1500]),
    (2, 8, 128, 128, 64, 0, [700], [1300]),
    (1, 2, 96, 96, 16, 0, [129], [4000]),
    (1, 8, 64, 64, 64, 0, [16] * 140, [5 * i for i in range(140)]),
    (2, 1, 192, 192, 64, 0, [384, 256], [0, 128]),
    (2, 4, 256, 256, 64, 0, [700, 33], [3000, 5000]),
    (3, 2, 136, 200, 16, 300, [900, 260], [1000, 0]),
    (4, 8, 128, 128, 32, 0, [513], [4000]),
]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
@pytest.mark.parametrize("dt,ct", TYPES)
def test_chunk(o1, dt, ct, case):
    G, hpg, d, dv, page, window, lens, pasts = CHUNKS[case]
    d, dv = unit(ct, d), unit(ct, dv)
    seqs, ends, rows = spread(lens, pasts, len(lens) + 1)
    g = o1.pg_geom(G, hpg, d, dv, page, dtype=dt, cache_dtype=ct, window=window)
    cache = Cache(o1, g, ends, 100 + case)
    q = randn(torch.Generator().manual_seed(case), rows, G * hpg, d, dtype=dt)
    q[0], q[-2:] = NAN, float("inf")      # rows of no sequence
    out = torch.full((rows, G * hpg, dv), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, seqs, out)
    check(o1, cache, q, seqs, out, f"case {case}")


# G, hpg, d, dv, page, window, positions
TOKENS = [
    (1, 1, 64, 64, 16, 0, [0]),
    (2, 4, 256, 256, 64, 0, [8190]),
    (2, 4, 128, 128, 16, 0, [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000, 5000, 3, 2047]),
    (4, 3, 72, 40, 32, 0, [300, 77, 1500]),
    (1, 16, 128, 64, 256, 0, [255, 256, 4095]),
    (3, 8, 64, 128, 64, 100, [99, 100, 101, 700, 3000, 0]),
    (1, 2, 200, 200, 128, 1, [0, 600, 128]),
    (8, 1, 32, 32, 16, 0, [(37 * i) % 700 for i in range(130)]),
    (1, 5, 8, 256, 16, 33, [40, 32, 31, 2000]),
    (2, 2, 256, 8, 16, 0, [31, 450]),
]


@pytest.mark.parametrize("case", range(len(TOKENS)))
@pytest.mark.parametrize("dt,ct", TYPES)
def test_token(o1, dt, ct, case):
    G, hpg, d, dv, page, window, at = TOKENS[case]
    d, dv = unit(ct, d), unit(ct, dv)
    n = len(at)
    g = o1.pg_geom(G, hpg, d, dv, page, dtype=dt, cache_dtype=ct, window=window)
    cache = Cache(o1, g, [p + 1 for p in at] + [7], 200 + case)
    gen = torch.Generator().manual_seed(case)
    # rows in another order than their slots, a padding row by slot, by position, and past the table
    order = torch.randperm(n, generator=gen).tolist()
    slots = [-1] + order + [n + 1, 0, 0]
    pos = [5] + [at[i] for i in order] + [0, -1, cache.table.shape[1] * page]
    q = randn(gen, n + 4, G * hpg, d, dtype=dt)
    q[0], q[-3:] = NAN, float("inf")
    out = torch.full((n + 4, G * hpg, dv), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, None, out, token=(torch.tensor(slots, dtype=torch.int32, device="cuda"), torch.tensor(pos, device="cuda")))
    check(o1, cache, q, [(r + 1, 1, i, at[i]) for r, i in enumerate(order)], out, f"case {case}")


@pytest.mark.parametrize("ct", [BF16, E4])
@pytest.mark.parametrize("d", [128, 256])
def test_fp32_rows_keep_fp32(o1, ct, d):
    """In the 2-norm fp32 outputs are near fp32's own error: the products of
    scores and values are of d and n terms, u sqrt(d) and u sqrt(n) at most
    each, with a handful of roundings: 16 u (2^-20) for the lengths here."""
    g = o1.pg_geom(2, 4, d, d, 64, dtype=F32, cache_dtype=ct)
    cache = Cache(o1, g, [6000], 9)
    q = randn(torch.Generator().manual_seed(4), 200, 8, d)
    seqs = [(0, 200, 0, 5800)]
    k, v = cache.held()
    want, _ = ref.attend(q, k, v, cache.table, 64, cache.n, seqs, g.scale, 0, F32, 3, 0.0)
    for form in ("chunk", "token"):
        out = torch.full((200, 8, d), NAN, device="cuda")
        attend(o1, cache, q, seqs, out, token=None if form == "chunk" else
               (torch.zeros(200, dtype=torch.int32, device="cuda"), torch.arange(5800, 6000, device="cuda")))
        err = float((out.double() - want).norm() / want.norm())
        print(form, err)
        assert err < 2.0 ** -20


@pytest.mark.parametrize("dt,ct", [(F32, BF16), (BF16, E4), (F16, F16)])
def test_extreme_scores(o1, dt, ct):
    """Scores of hundreds: one position carries a row, the reference moves often,
    and rows' first positions are far below the later ones."""
    g = o1.pg_geom(1, 2, 64, 64, 16, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, [700], 11)
    n = torch.arange(700, device="cuda")
    ids, at = ref.places(cache.table, 16, 0, 0, 700)
    if ct is E4:
        cache.ke[ids, 0, at] = (110 + (n * 7) % 20).to(torch.uint8)
    else:
        cache.k[ids, 0, at] *= torch.exp2(((n * 7) % 10 - 4).float())[:, None].to(ct)
    q = (randn(torch.Generator().manual_seed(5), 700, 2, 64) * 4).to(dt)
    out = torch.full((700, 2, 64), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, [(0, 700, 0, 0)], out)
    check(o1, cache, q, [(0, 700, 0, 0)], out, "chunk")
    out = torch.full((700, 2, 64), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, None, out, token=(torch.zeros(700, dtype=torch.int32, device="cuda"), n))
    check(o1, cache, q, [(r, 1, 0, r) for r in range(700)], out, "rows")


@pytest.mark.parametrize("dt,ct", TYPES)
@pytest.mark.parametrize("hpg,d", [(1, 64), (2, 144)])
def test_non_finite_rows_spoil_only_what_is_near(o1, dt, ct, hpg, d):
    """A key that is infinite and a value that is NaN: rows 384 and more before
    them and the other sequence are as if they were not there, rows from the
    value's position on are NaN."""
    at, lens = 700, [1000, 150]
    g = o1.pg_geom(1, hpg, d, d, 64, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, lens, 31)
    for pool, value in ((cache.v, NAN), (cache.k, float("inf"))):
        ids, n = ref.places(cache.table, 64, 0, at, at + 1)
        if ct is E4:
            pool.view(torch.uint8)[ids, 0, n] = 0x7f
        else:
            pool[ids, 0, n] = value
        q = randn(torch.Generator().manual_seed(6), sum(lens), hpg, d, dtype=dt)
        out = torch.zeros(sum(lens), hpg, d, dtype=dt, device="cuda")
        attend(o1, cache, q, [(0, lens[0], 0, 0), (lens[0], lens[1], 1, 0)], out)
        seqs = [(0, at - 383, 0, 0), (lens[0], lens[1], 1, 0)]
        k, v = cache.held()
        terms, rho, f16 = ref.precision(dt, ct)
        want, bound = ref.attend(q, k, v, cache.table, 64, cache.n, seqs, g.scale, 0, dt, terms, rho, f16, cache.ve)
        for r0, n, _, _ in seqs:
            ref.assert_within(out[r0:r0 + n], want[r0:r0 + n].cpu(), bound[r0:r0 + n].cpu(), f"rows {r0} on")
        assert torch.isnan(out[at:lens[0]]).all()


@pytest.mark.parametrize("dt,ct", [(F32, BF16), (BF16, E4)])
def test_strides_and_slices(o1, dt, ct):
    """q, k, v as columns of one projection's rows; out as columns of a buffer;
    a layer's cache as a slice of a pool of several layers."""
    G, hpg, d, page, rows = 2, 3, 64, 32, 100
    g = o1.pg_geom(G, hpg, d, d, page, dtype=dt, cache_dtype=ct)
    gen = torch.Generator().manual_seed(6)
    qkv = randn(gen, rows, (G * hpg + 2 * G) * d + 16, dtype=dt)
    q = qkv[:, :G * hpg * d].unflatten(1, (G * hpg, d))
    k = qkv[:, G * hpg * d:G * (hpg + 1) * d].unflatten(1, (G, d))
    v = qkv[:, G * (hpg + 1) * d:G * (hpg + 2) * d].unflatten(1, (G, d))
    cache = Cache(o1, g, [rows], 13)
    pools = [torch.zeros(3, *x.shape, dtype=torch.uint8, device="cuda").repeat_interleave(x.element_size(), -1).view(x.dtype)
             for x in (cache.k, cache.v)]
    exps = [torch.ones(3, *x.shape, dtype=torch.uint8, device="cuda") if x is not None else None for x in (cache.ke, cache.ve)]
    cache.k, cache.v = pools[0][1], pools[1][1]
    cache.ke, cache.ve = (x[1] if x is not None else None for x in exps)
    cache.c = o1.pg_cache(g, cache.k, cache.v, cache.table, cache.ke, cache.ve)
    wide = torch.full((rows, 3 * G * hpg * d), NAN, dtype=dt, device="cuda")
    out = wide[:, G * hpg * d:2 * G * hpg * d].unflatten(1, (G * hpg, d))
    o1.check(o1.o1_pg_write(g, cache.c, k, v, [(0, rows, 0, 0)]), "write")
    attend(o1, cache, q, [(0, rows, 0, 0)], out)
    check(o1, cache, q, [(0, rows, 0, 0)], out, "strides")
    assert torch.isnan(wide[:, :G * hpg * d]).all() and torch.isnan(wide[:, 2 * G * hpg * d:]).all()
    assert all((x[i].view(torch.uint8) == 0).all() for x in pools for i in (0, 2))


@pytest.mark.parametrize("dt,ct", [(BF16, BF16), (F16, E4)])
def test_most_rows(o1, dt, ct):
    """65536 decode rows, written and attended in a call each; some of them checked."""
    n = 65536
    g = o1.pg_geom(1, 2, 16, 16, 16, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, [2 + r % 40 for r in range(n)], 41)
    gen = torch.Generator().manual_seed(42)
    k, v, q = (randn(gen, n, h, 16, dtype=dt) for h in (1, 1, 2))
    pos = torch.arange(n, device="cuda") % 40 + 1
    o1.check(o1.o1_pg_token_write(g, cache.c, k, v, None, pos), "write")
    out = torch.full((n, 2, 16), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, None, out, token=(None, pos))
    some = list(range(0, n, 409)) + [n - 2, n - 1]
    held = ref.quantise(k)[0] if ct is E4 else k.double()
    for r in some[::10]:
        ids, at = ref.places(cache.table, 16, r, int(pos[r]), int(pos[r]) + 1)
        assert torch.equal(ref.held(cache.k, cache.ke)[ids, :, at][0], held[r])
    seqs = [(r, 1, r, int(pos[r])) for r in some]
    terms, rho, f16 = ref.precision(dt, ct)
    want, bound = ref.attend(q, *cache.held(), cache.table, 16, cache.n, seqs, g.scale, 0, dt, terms, rho, f16, cache.ve)
    ref.assert_within(out[some], want[some].cpu(), bound[some].cpu(), "rows")
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dt,ct", [(BF16, BF16), (BF16, E4), (F32, BF16)])
@pytest.mark.parametrize("hpg", [4, 16])
def test_most_sequences(o1, dt, ct, hpg):
    """4096 sequences of 3 rows, in 32 launches over the same scratch."""
    n = 4096
    g = o1.pg_geom(1, hpg, 32, 32, 16, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, [3 + r % 60 for r in range(n)], 43)
    q = randn(torch.Generator().manual_seed(44), 3 * n, hpg, 32, dtype=dt)
    out = torch.full((3 * n, hpg, 32), NAN, dtype=dt, device="cuda")
    seqs = [(3 * r, 3, r, r % 60) for r in range(n)]
    attend(o1, cache, q, seqs, out)
    some = seqs[::31] + seqs[-1:]
    terms, rho, f16 = ref.precision(dt, ct)
    want, bound = ref.attend(q, *cache.held(), cache.table, 16, cache.n, some, g.scale, 0, dt, terms, rho, f16, cache.ve)
    rows = [r0 + i for r0, m, _, _ in some for i in range(m)]
    ref.assert_within(out[rows], want[rows].cpu(), bound[rows].cpu(), "sequences")
    assert torch.isfinite(out).all()


def test_far_offsets(o1):
    """A cache whose offsets pass 2^31 values: its last pages, 2.3 GB in."""
    G, d, page = 2, 256, 256
    g = o1.pg_geom(G, 2, d, 16, page, dtype=BF16, cache_dtype=E4)
    n = (2 ** 31 + 2 ** 28) // (G * page * d)
    k, v = torch.zeros(n, G, page, d, dtype=E4, device="cuda"), torch.zeros(n, G, page, 16, dtype=E4, device="cuda")
    ke, ve = (torch.full((n, G, page), 120, dtype=torch.uint8, device="cuda") for _ in "kv")
    table = torch.tensor([[n - 1, 0, n - 2]], dtype=torch.int32, device="cuda")
    c = o1.pg_cache(g, k, v, table, ke, ve)
    gen = torch.Generator().manual_seed(7)
    rows = 700
    kk, vv, q = randn(gen, rows, G, d, dtype=BF16), randn(gen, rows, G, 16, dtype=BF16), randn(gen, rows, 4, d, dtype=BF16)
    o1.check(o1.o1_pg_write(g, c, kk, vv, [(0, rows, 0, 0)]), "write")
    bk, bv = torch.zeros_like(kk), torch.zeros_like(vv)
    o1.check(o1.o1_pg_read(g, c, [(0, rows, 0, 0)], bk, bv), "read")
    assert torch.equal(bk.double(), ref.quantise(kk)[0]) and torch.equal(bv.double(), ref.quantise(vv)[0])
    scratch = torch.empty(o1.o1_pg_scratch_bytes(g, rows), dtype=torch.uint8, device="cuda")
    out, one = torch.zeros(rows, 4, 16, dtype=BF16, device="cuda"), torch.zeros(1, 4, 16, dtype=BF16, device="cuda")
    o1.check(o1.o1_pg_chunk_attend(g, c, scratch, q, [(0, rows, 0, 0)], out), "chunk")
    o1.check(o1.o1_pg_token_attend(g, c, scratch, q[-1:], None, torch.tensor([rows - 1], device="cuda"), one), "token")
    near = lambda x: ref.quantise(x)[0].unflatten(0, (1, rows)).transpose(1, 2)   # one page of all the rows
    exp = ref.quantise(vv)[1].unflatten(0, (1, rows)).transpose(1, 2)
    want, bound = ref.attend(q, near(kk), near(vv), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), rows, 1, [(0, rows, 0, 0)],
                             g.scale, 0, BF16, *ref.precision(BF16, E4), v_exp=exp)
    ref.assert_within(out, want.cpu(), bound.cpu(), "far chunk")
    ref.assert_within(one, want[-1:].cpu(), bound[-1:].cpu(), "far row")


def test_capture_and_replay(o1):
    """A decode step of write and attention, captured once and replayed as the
    sequences grow and change places, between calls of other sizes that share
    the scratch."""
    G, hpg, d, page = 2, 4, 64, 16
    g = o1.pg_geom(G, hpg, d, d, page, dtype=BF16, cache_dtype=E4)
    cache = Cache(o1, g, [2000, 300, 50], 17)
    gen = torch.Generator().manual_seed(8)
    scratch = torch.empty(o1.o1_pg_scratch_bytes(g, 64), dtype=torch.uint8, device="cuda")
    k, v, q = (torch.zeros(3, h, d, dtype=BF16, device="cuda") for h in (G, G, G * hpg))
    out = torch.full((3, G * hpg, d), NAN, dtype=BF16, device="cuda")
    slots, pos = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")

    def step():
        o1.check(o1.o1_pg_token_write(g, cache.c, k, v, slots, pos), "write")
        o1.check(o1.o1_pg_token_attend(g, cache.c, scratch, q, slots, pos, out), "attend")

    slots.copy_(torch.tensor([0, 1, -1]))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for at in ([(0, 700), (1, 299), (2, 0)], [(2, 49), (0, 1999), (-1, 0)], [(1, 3), (0, 1800), (2, 20)]):
        slots.copy_(torch.tensor([s for s, _ in at]))
        pos.copy_(torch.tensor([p for _, p in at]))
        for x in (k, v, q):
            x.copy_(randn(gen, *x.shape, dtype=BF16))
        out.fill_(NAN)
        graph.replay()
        check(o1, cache, q, [(r, 1, s, p) for r, (s, p) in enumerate(at) if s >= 0], out, f"replay {at}")
        big = randn(gen, 64, G * hpg, d, dtype=BF16)
        bout = torch.full((64, G * hpg, d), NAN, dtype=BF16, device="cuda")
        o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, big, [(0, 64, 0, 1900)], bout), "chunk")
        check(o1, cache, big, [(0, 64, 0, 1900)], bout, "chunk on the same scratch")


def test_chunk_in_a_graph_and_on_other_streams(o1):
    G, hpg, d, page = 2, 2, 128, 64
    g = o1.pg_geom(G, hpg, d, d, page, dtype=BF16)
    seqs, ends, rows = spread([300, 5], [100, 900], 3)
    cache = Cache(o1, g, ends, 19)
    q = randn(torch.Generator().manual_seed(9), rows, G * hpg, d, dtype=BF16)
    outs = [torch.full((rows, G * hpg, d), NAN, dtype=BF16, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    kept = [attend(o1, cache, q, seqs, o, stream=s) for s, o in zip(streams, outs)]   # at once, a scratch each
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    scratch = kept[0]
    with torch.cuda.graph(graph):
        o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, q, seqs, outs[2]), "chunk")
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        check(o1, cache, q, seqs, o, "stream")
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16)), "results differ from call to call"


def test_binding_refusals(o1):
    g = o1.pg_geom(2, 2, 64, 32, 16, dtype=F32)
    cache = Cache(o1, g, [40], 21)
    q, out = torch.zeros(4, 4, 64, device="cuda"), torch.zeros(4, 4, 32, device="cuda")
    k, v = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, 2, 32, device="cuda")
    scratch = torch.empty(o1.o1_pg_scratch_bytes(g, 4), dtype=torch.uint8, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    ok = lambda **kw: o1.o1_pg_token_attend(kw.get("g", g), cache.c, scratch, kw.get("q", q), kw.get("slots"), kw.get("pos", pos[:1]),
                                            kw.get("out", out))
    for bad, err in ((dict(q=q.half()), TypeError), (dict(q=q.cpu()), TypeError), (dict(q=q[:, :3]), ValueError), (dict(out=out[:3]), ValueError),
                     (dict(pos=pos.int()), TypeError), (dict(pos=pos[:3]), ValueError), (dict(slots=pos), TypeError),
                     (dict(q=q.transpose(0, 1)), ValueError), (dict(g=o1.pg_geom(2, 2, 64, 32, 32)), ValueError)):
        with pytest.raises(err):
            ok(**bad)
    with pytest.raises(TypeError):
        o1.o1_pg_write(g, cache.c, k.bfloat16(), v, [(0, 4, 0, 0)])
    for bad, err in (((cache.k, cache.v[:1], cache.table), ValueError), ((cache.k.float(), cache.v, cache.table), TypeError),
                     ((cache.k, cache.v, cache.table.long()), TypeError), ((cache.k, cache.v, cache.table[0]), ValueError),
                     ((cache.k, cache.v, None), TypeError), ((cache.k, cache.v, cache.table, cache.k), ValueError)):
        with pytest.raises(err):
            o1.pg_cache(g, *bad)
    assert o1.o1_pg_chunk_attend(g, cache.c, scratch[:256], q, [(0, 4, 0, 0)], out) == o1.O1_ERR_ARG
    assert o1.o1_pg_write(g, cache.c, k, v, [(0, 4, 1, 0)]) == o1.O1_ERR_ARG
    torch.cuda.synchronize()


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("dt,ct", [(F32, E4), (BF16, BF16), (F16, F16)])
def test_prompt_then_decode(o1, dt, ct):
    """Two sequences as a model serves them: heads normalised and rotated, prompt
    written and attended, then rows one at a time; every row equals the
    attention of the whole sequence in one call."""
    G, hpg, d, page, n = 2, 4, 64, 16, 90
    g = o1.pg_geom(G, hpg, d, d, page, dtype=dt, cache_dtype=ct)
    cache = Cache(o1, g, [n, n], 23, fill=False)
    gen = torch.Generator().manual_seed(10)
    raw = [randn(gen, 2 * n, h, d, dtype=dt) for h in (G * hpg, G, G)]
    inv = (1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    prep = o1.prep_geom(G * hpg, G, d, in_dtype=dt)
    scratch = torch.empty(o1.o1_pg_scratch_bytes(g, 2 * n), dtype=torch.uint8, device="cuda")
    out = torch.full((2 * n, G * hpg, d), NAN, dtype=dt, device="cuda")
    place = torch.arange(n, device="cuda").repeat(2)
    q, k, v = raw[0].clone(), raw[1].clone(), raw[2]
    o1.check(o1.o1_head_prep(prep, q, k, None, None, inv, q, k, pos=place), "prep")
    first = [61, 33]
    seqs = [(0, first[0], 0, 0), (n, first[1], 1, 0)]
    o1.check(o1.o1_pg_write(g, cache.c, k, v, seqs), "write")
    o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, q, seqs, out), "chunk")
    slots, pos = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), torch.tensor([first[1], first[0]], device="cuda")
    for step in range(n - first[1]):
        rows = [n + first[1] + step, first[0] + step if first[0] + step < n else 0]
        if first[0] + step >= n:
            slots[1] = -1      # done: padding
        x = [t[rows].contiguous() for t in raw]
        o1.check(o1.o1_head_prep(prep, x[0], x[1], None, None, inv, x[0], x[1], pos=pos), "prep")
        o1.check(o1.o1_pg_token_write(g, cache.c, x[1], x[2], slots, pos), "write")
        got = torch.full((2, G * hpg, d), NAN, dtype=dt, device="cuda")
        o1.check(o1.o1_pg_token_attend(g, cache.c, scratch, x[0], slots, pos, got), "attend")
        out[rows[0]] = got[0]
        if first[0] + step < n:
            out[rows[1]] = got[1]
        else:
            assert torch.isnan(got[1]).all()
        pos += 1
    # what was cached is what a write of the whole holds
    for x, pool, exp in ((k, cache.k, cache.ke), (v, cache.v, cache.ve)):
        for s in range(2):
            ids, at = ref.places(cache.table, page, s, 0, n)
            want = ref.quantise(x[s * n:(s + 1) * n])[0] if ct is E4 else x[s * n:(s + 1) * n].to(ct).double()
            assert torch.equal(ref.held(pool, exp)[ids, :, at], want)
    check(o1, cache, q, [(0, n, 0, 0), (n, n, 1, 0)], out, "prompt and decode")


def test_sealing_from_the_cache(o1):
    """An exact layer's cache moves a sealed layer over its rows: read back as
    fp32 rows into o1_spec_commit, the state is that of the rows themselves."""
    import harness
    from sliding_window_landmark_gb300 import synth
    sh = synth.Shape(groups=2, heads_per_group=2, d=64, dv=64, sinks=4, window=64, landmarks=8)
    c = synth.layer_constants(sh, 3)
    rows = 150
    gen = torch.Generator().manual_seed(12)
    k, v = randn(gen, rows, 2, 64, dtype=BF16).float(), randn(gen, rows, 2, 64, dtype=BF16).float()
    g = o1.pg_geom(2, 2, 64, 64, 32, dtype=F32)      # bf16 values: held exactly
    cache = Cache(o1, g, [rows], 25)
    o1.check(o1.o1_pg_write(g, cache.c, k, v, [(0, rows, 0, 0)]), "write")
    bk, bv = torch.zeros_like(k), torch.zeros_like(v)
    o1.check(o1.o1_pg_read(g, cache.c, [(0, rows, 0, 0)], bk, bv), "read")
    assert torch.equal(bk, k) and torch.equal(bv, v)
    states = []
    for kk, vv in ((k, v), (bk, bv)):
        lay = harness.GpuLayer(sh, c, max_rows=rows)
        o1.check(o1.o1_spec_commit(lay.state, lay.g, lay.scratch, kk, vv, rows), "commit")
        states.append(lay.read())
    for name in states[0]:
        assert (states[0][name] == states[1][name]).all(), name


@pytest.mark.parametrize("dt,ct,d", [(BF16, BF16, 128), (BF16, E4, 256), (F32, BF16, 64), (F16, E4, 128)])
def test_expired_waits_leave_nan_or_right_values(o1, dt, ct, d):
    """The waits of the tensor-core kernel run out on purpose, early and at
    several points: a flag, every value NaN or right, and the next call is right."""
    g = o1.pg_geom(2, 4, d, d, 64, dtype=dt, cache_dtype=ct)
    seqs = [(0, 300, 0, 600), (300, 100, 1, 0)]
    cache = Cache(o1, g, [900, 100], 27)
    q = randn(torch.Generator().manual_seed(13), 400, 8, d, dtype=dt)
    k, v = cache.held()
    want, bound = ref.attend(q, k, v, cache.table, 64, cache.n, seqs, g.scale, 0, dt, *ref.precision(dt, ct), v_exp=cache.ve)
    assert o1.o1_pg_flags(clear=True) == 0
    raised = 0
    for limit in (1, 300, 1000, 2000, 3000, 5000, 8000, 20000):
        out = torch.full((400, 8, d), 77.0, dtype=dt, device="cuda")
        try:
            o1.o1_set_wait_limit(limit)
            attend(o1, cache, q, seqs, out)
        finally:
            o1.o1_set_wait_limit(0)
        flags = o1.o1_pg_flags(clear=True)
        raised += flags == o1.O1_FLAG_WAIT_EXPIRED
        bad = ~torch.isnan(out) & ((out.double() - want).abs() > bound)
        assert not bad.any(), f"limit {limit}: {int(bad.sum())} values neither NaN nor right"
        assert flags or torch.isfinite(out).all()
    assert raised and o1.o1_pg_flags() == 0
    out = torch.full((400, 8, d), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, seqs, out)
    check(o1, cache, q, seqs, out, "after expiry")
    assert o1.o1_pg_flags() == 0


@pytest.mark.parametrize("dt,ct,d", [(BF16, BF16, 128), (F16, F16, 256), (BF16, E4, 128), (F32, E4, 64), (F32, BF16, 64)])
def test_calls_behind_expired_waits_are_right(o1, dt, ct, d):
    """Blocks whose waits ran out at once, with their first copies on the way and no
    wait of the senders among them, keep their shared memory until the copies have
    landed: calls directly behind them, whose blocks take that memory, are right,
    and the same bit for bit."""
    g = o1.pg_geom(2, 4, d, d, 64, dtype=dt, cache_dtype=ct)
    seqs = [(0, 256, 0, 640), (256, 64, 1, 64)]
    cache = Cache(o1, g, [896, 128], 29)
    q = randn(torch.Generator().manual_seed(14), 320, 8, d, dtype=dt)
    scratch = torch.empty(o1.o1_pg_scratch_bytes(g, 320), dtype=torch.uint8, device="cuda")
    slots, pos = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([895, 127], device="cuda")
    lost = torch.empty(320, 8, d, dtype=dt, device="cuda")
    outs = [torch.full((322, 8, d), NAN, dtype=dt, device="cuda") for _ in range(24)]
    o1.o1_pg_flags(clear=True)
    for out in outs:
        try:
            o1.o1_set_wait_limit(1)
            o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, q, seqs, lost), "expired")
        finally:
            o1.o1_set_wait_limit(0)
        o1.check(o1.o1_pg_token_attend(g, cache.c, scratch, q[255:320:64], slots, pos, out[320:]), "token")
        o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, q, seqs, out[:320]), "chunk")
    assert o1.o1_pg_flags(clear=True) == o1.O1_FLAG_WAIT_EXPIRED
    check(o1, cache, q, seqs, outs[0][:320], "chunk behind expired waits")
    check(o1, cache, q[255:320:64], [(0, 1, 0, 895), (1, 1, 1, 127)], outs[0][320:], "rows behind expired waits")
    for out in outs[1:]:
        assert torch.equal(out.view(torch.uint8), outs[0].view(torch.uint8)), "results differ from call to call"


@pytest.mark.parametrize("dt,ct,d", [(BF16, BF16, 128), (F16, F16, 256), (F32, BF16, 128), (F32, BF16, 64), (BF16, E4, 128), (F16, E4, 256)])
def test_expired_waits_in_long_shares(o1, dt, ct, d):
    """Waits that run out late: blocks of several units and many tiles, most of them
    whole (boxes), of one and of two query tiles, whose rings are around more than
    once. Every value is NaN or right, a call without the flag is right, and every
    call ends soon: a block that waited for a phase that does not come would take
    4e9 cycles, 1.9 s at the highest clock, where a call takes less than a millisecond."""
    import time
    g = o1.pg_geom(2, 4, d, d, 64, dtype=dt, cache_dtype=ct)
    rows = [(64, 32, 300)[i % 3] for i in range(60)]
    ends = [(1024, 896, 1280)[i % 3] + (i % 7 == 0) * 5 for i in range(60)]
    seqs, at = [], 0
    for i, (n, end) in enumerate(zip(rows, ends)):
        seqs.append((at, n, i, end - n))
        at += n
    cache = Cache(o1, g, ends, 31)
    q = randn(torch.Generator().manual_seed(15), at, 8, d, dtype=dt)
    k, v = cache.held()
    want, bound = ref.attend(q, k, v, cache.table, 64, cache.n, seqs, g.scale, 0, dt, *ref.precision(dt, ct), v_exp=cache.ve)
    out = torch.full((at, 8, d), NAN, dtype=dt, device="cuda")
    scratch = attend(o1, cache, q, seqs, out)
    ref.assert_within(out, want.cpu(), bound.cpu(), "without limits")
    assert o1.o1_pg_flags(clear=True) == 0
    raised = []
    for limit in (1, 500, 1000, 1500, 2000, 2500, 3000, 3500, 4000, 5000, 6000, 8000, 12000, 20000, 40000):
        for _ in range(3):
            out.fill_(77.0)
            torch.cuda.synchronize()
            start = time.perf_counter()
            try:
                o1.o1_set_wait_limit(limit)
                o1.check(o1.o1_pg_chunk_attend(g, cache.c, scratch, q, seqs, out), "chunk")
            finally:
                o1.o1_set_wait_limit(0)
            flags = o1.o1_pg_flags(clear=True)
            took = time.perf_counter() - start
            assert took < 0.5, f"limit {limit}: {took} s"
            bad = ~torch.isnan(out) & ((out.double() - want).abs() > bound)
            assert not bad.any(), f"limit {limit}: {int(bad.sum())} values neither NaN nor right"
            assert flags or torch.isfinite(out).all()
            raised.append((limit, flags, float(torch.isnan(out).double().mean())))
    assert any(f == o1.O1_FLAG_WAIT_EXPIRED for _, f, _ in raised)
    print("limit, flags and part of NaN:", raised)
    attend(o1, cache, q, seqs, out)
    ref.assert_within(out, want.cpu(), bound.cpu(), "after expiry")
    assert o1.o1_pg_flags() == 0


@pytest.mark.parametrize("dt,ct,d,rows", [(F16, F16, 64, 1), (F16, F16, 128, 64), (F16, F16, 256, 40), (F16, F16, 256, 2), (BF16, E4, 64, 1),
                                          (F16, E4, 128, 1), (BF16, E4, 256, 2), (F16, E4, 64, 64), (BF16, E4, 128, 64)])
def test_small_weights_under_a_large_one(o1, dt, ct, d, rows):
    """The output is the sum of a thousand small weights beside one large one that
    adds nothing to it: a key 15.3 above the others in score (weights of 2^-22 of
    the largest) whose value is 0, or, over e4m3, a value row 2^24 times as large
    whose other columns are 0. Weights held in fp16 may be off by 2^-11 of their
    value and 2^-32 of the largest (over e4m3, of weights times their values' powers
    of two), as the header states; the reference's bound counts 2^-25 for the latter,
    so that its part is taken 2^-7 times."""
    G, hpg, page, past = 2, 4, 64, 1000
    g = o1.pg_geom(G, hpg, d, d, page, dtype=dt, cache_dtype=ct)
    n = past + rows
    cache = Cache(o1, g, [n], 33, fill=False)
    gen = torch.Generator().manual_seed(16)
    q = randn(gen, rows, G * hpg, d) * 0.25
    k = randn(gen, n, G, d) * 0.05
    v = 500 + 500 * torch.rand(n, G, d, generator=gen).cuda()
    q[..., 0], k[..., 0] = 4.0, 0.0
    if ct is E4:
        v *= 2.0 ** -19                      # under 2^-17, the large row under 2^7
        k[3, :, 0], v[3] = 0.065 * d ** 0.5, 0.0
        v[3, :, 5] = 440 * 2.0 ** 7
    else:
        k[3, :, 0], v[3] = 15.3 / 4 * d ** 0.5, 0.0
    q, k, v = (x.to(dt) for x in (q, k, v))
    o1.check(o1.o1_pg_write(g, cache.c, k, v, [(0, n, 0, 0)]), "write")
    seqs = [(0, rows, 0, past)]
    out = torch.full((rows, G * hpg, d), NAN, dtype=dt, device="cuda")
    attend(o1, cache, q, seqs, out)
    terms, rho, f16 = ref.precision(dt, ct)
    if f16 and rows * hpg <= 16:
        rho = 2.0 ** -11                     # few rows over e4m3: fp16 for bf16 rows too
    args = (q, *cache.held(), cache.table, page, cache.n, seqs, g.scale, 0, dt, terms, rho)
    want, bound = ref.attend(*args, False, cache.ve)
    coarse = ref.attend(*args, True, cache.ve)[1]
    ref.assert_within(out, want.cpu(), (bound + 2.0 ** -7 * (coarse - bound)).cpu(), "small weights")


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("dt,ct,d", [(F32, BF16, 256), (F32, E4, 256), (BF16, E4, 128), (F16, F16, 64)])
def test_launches_hold_what_a_table_admits(o1, dt, ct, d, window):
    """A call launches the blocks that its table's width (or its sequences) can
    give a share to. The split of the keys depends on the lengths alone, so that a
    wide table and a narrow one, a chunk of one row and a token give the same bits; a
    call of one block alone is right."""
    G, hpg, page = 2, 4, 16
    g = o1.pg_geom(G, hpg, d, d, page, dtype=dt, cache_dtype=ct, window=window)
    ends = [1, 64, 65, 400, 799, 800]
    cache = Cache(o1, g, ends, 35)
    gen = torch.Generator().manual_seed(17)
    wide = torch.full((len(ends), 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, :50] = cache.table[:, :50]
    tables = {"narrow": wide[:, :50].contiguous(), "wide": wide}
    for rows in ([0], [3], [5], list(range(6))):
        q = randn(gen, len(rows), G * hpg, d, dtype=dt)
        seqs = [(i, 1, s, ends[s] - 1) for i, s in enumerate(rows)]
        slots = torch.tensor(rows, dtype=torch.int32, device="cuda")
        pos = torch.tensor([ends[s] - 1 for s in rows], device="cuda")
        outs = []
        for table in tables.values():
            cache.c = o1.pg_cache(g, cache.k, cache.v, table, cache.ke, cache.ve)
            for token in ((slots, pos), None):
                outs.append(torch.full((len(rows), G * hpg, d), NAN, dtype=dt, device="cuda"))
                attend(o1, cache, q, seqs, outs[-1], token=token)
        check(o1, cache, q, seqs, outs[0], f"rows {rows}")
        for o in outs[1:]:
            assert torch.equal(o.view(torch.uint8), outs[0].view(torch.uint8)), f"rows {rows}"
