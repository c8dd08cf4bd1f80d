"""The paged cache without a GPU: sizes, the refusals of the entry points' C
checks, which come before any CUDA call, and those of the binding."""
import ctypes

import pytest
import torch

import pg_reference as ref

V = ctypes.c_void_p
MB = 1 << 20
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def o1():
    from sliding_window_landmark_gb300 import build
    build.build()
    from sliding_window_landmark_gb300 import o1 as mod
    return mod


def geom(o1, **kw):
    return o1.pg_geom(kw.pop("G", 2), kw.pop("hpg", 2), kw.pop("d", 64), kw.pop("dv", 32), kw.pop("page", 16), **kw)


def cache(o1, **kw):
    c = dict(k=128 * MB, v=144 * MB, k_exp=160 * MB, v_exp=161 * MB, table=162 * MB, n_pages=8, n_slots=4, width=4)
    c.update(kw)
    return o1.o1_pg_cache(*[c[n] for n in ("k", "v", "k_exp", "v_exp", "table", "n_pages", "n_slots", "width")])


def ref_or_none(x):
    return ctypes.byref(x) if x is not None else None


def write(o1, g=None, c=0, k=MB, ks=128, v=2 * MB, vs=64, seqs=((0, 4, 0, 0),), rows=8, fn="o1_pg_write"):
    g = g or geom(o1)
    arr = o1.pg_seqs(seqs) if seqs is not None else None
    n = len(seqs) if seqs is not None else 1
    c = cache(o1) if c == 0 else c
    if fn == "o1_pg_write":
        return o1.LIB.o1_pg_write(ctypes.byref(g), ref_or_none(c), V(k), ks, V(v), vs, arr, n, rows, None)
    return o1.LIB.o1_pg_read(ctypes.byref(g), ref_or_none(c), arr, n, V(k), ks, V(v), vs, rows, None)


def chunk(o1, g=None, c=0, scratch=32 * MB, nbytes=32 * MB, q=MB, qs=256, seqs=((0, 4, 0, 0),), out=4 * MB, os_=128, rows=8):
    g = g or geom(o1)
    arr = o1.pg_seqs(seqs) if seqs is not None else None
    return o1.LIB.o1_pg_chunk_attend(ctypes.byref(g), ref_or_none(cache(o1) if c == 0 else c), V(scratch), nbytes, V(q), qs, arr,
                                     len(seqs) if seqs is not None else 1, V(out), os_, rows, None)


def token(o1, g=None, c=0, scratch=32 * MB, nbytes=32 * MB, q=MB, qs=256, slots=6 * MB, pos=7 * MB, out=4 * MB, os_=128, rows=4):
    g = g or geom(o1)
    return o1.LIB.o1_pg_token_attend(ctypes.byref(g), ref_or_none(cache(o1) if c == 0 else c), V(scratch), nbytes, V(q), qs,
                                     V(slots), V(pos), V(out), os_, rows, None)


def token_write(o1, g=None, c=0, k=MB, ks=128, v=2 * MB, vs=64, slots=6 * MB, pos=7 * MB, rows=4):
    g = g or geom(o1)
    return o1.LIB.o1_pg_token_write(ctypes.byref(g), ref_or_none(cache(o1) if c == 0 else c), V(k), ks, V(v), vs, V(slots), V(pos),
                                    rows, None)


def bad_geoms(o1):
    e4 = dict(cache_dtype=E4)
    bad = [geom(o1, G=0), geom(o1, G=4097), geom(o1, hpg=0), geom(o1, hpg=17), geom(o1, G=4096, hpg=16), geom(o1, d=4),
           geom(o1, d=60), geom(o1, d=264), geom(o1, dv=0), geom(o1, dv=264), geom(o1, d=72, **e4), geom(o1, dv=40, **e4),
           geom(o1, page=8), geom(o1, page=48), geom(o1, page=512), geom(o1, page=0), geom(o1, window=-1),
           geom(o1, scale=float("nan")), geom(o1, scale=float("inf")), geom(o1, scale=0.0),
           geom(o1, scale=-1.0), geom(o1, cache_dtype=HF), geom(o1, dtype=BF, cache_dtype=HF),
           geom(o1, dtype=HF, cache_dtype=BF)]
    for n in (-1, 3, 4):
        g = geom(o1)
        g.dtype = n
        bad.append(g)
    for n in (-1, 0, 4):
        g = geom(o1)
        g.cache_dtype = n
        bad.append(g)
    return bad


def test_geometries(o1):
    for g in bad_geoms(o1):
        assert o1.o1_pg_scratch_bytes(g, 1) == 0
        for call in (write, chunk, token, token_write, lambda o1, g: write(o1, g, fn="o1_pg_read")):
            assert call(o1, g=g) == o1.O1_ERR_UNSUPPORTED
    for g in (geom(o1), geom(o1, G=4095, hpg=16), geom(o1, d=8, dv=256), geom(o1, d=16, dv=16, cache_dtype=E4, page=256),
              geom(o1, dtype=HF, cache_dtype=HF, window=2 ** 31 - 1), geom(o1, dtype=HF, cache_dtype=E4)):
        assert o1.o1_pg_scratch_bytes(g, 0) == 0
        sizes = [o1.o1_pg_scratch_bytes(g, n) for n in (1, 2, 16, 100, 10 ** 5, 2 ** 31 - 1)]
        assert 0 < sizes[0] and sizes == sorted(sizes) and sizes[-1] < 128 * MB, sizes


def test_cache_refusals(o1):
    A = o1.O1_ERR_ARG
    e4 = geom(o1, cache_dtype=E4)
    for call in (write, chunk, token, token_write, lambda o1, **kw: write(o1, fn="o1_pg_read", **kw)):
        assert call(o1, c=None) == A
        for name in ("k", "v", "table"):
            assert call(o1, c=cache(o1, **{name: None})) == A, name
            assert call(o1, c=cache(o1, **{name: 128 * MB + 8})) == A, name
        for name in ("k_exp", "v_exp"):
            assert call(o1, g=e4, c=cache(o1, **{name: None})) == A, name
            assert call(o1, c=cache(o1, **{name: 160 * MB + 8})) == A, name
        for name in ("n_pages", "n_slots", "width"):
            assert call(o1, c=cache(o1, **{name: 0})) == A, name
            assert call(o1, c=cache(o1, **{name: -1})) == A, name
        assert call(o1, c=cache(o1, n_pages=2 ** 26)) == A       # 2 groups of 16: 2^31 rows
        assert call(o1, c=cache(o1, width=2 ** 27)) == A
    # a write's pools over one another, over the table, over the exponents
    for call in (write, token_write):
        for over in (dict(v=128 * MB), dict(v=128 * MB + 64), dict(table=144 * MB)):
            assert call(o1, c=cache(o1, **over)) == A, over
        assert call(o1, g=e4, c=cache(o1, v_exp=160 * MB)) == A
        assert call(o1, g=e4, c=cache(o1, k_exp=162 * MB)) == A


SEQ_BAD = (((-1, 4, 0, 0),), ((0, -1, 0, 0),), ((0, 9, 0, 0),), ((5, 4, 0, 0),), ((0, 4, 4, 0),), ((0, 4, -1, 0),), ((0, 4, 0, -1),),
           ((0, 4, 0, 61),), ((0, 4, 0, 2 ** 31 - 1),), ((0, 4, 0, 0), (3, 2, 1, 0)), ((4, 4, 0, 0), (0, 5, 1, 0)),
           ((2 ** 31 - 1, 2 ** 31 - 1, 0, 0),))


def test_copy_refusals(o1):
    A = o1.O1_ERR_ARG
    for fn in ("o1_pg_write", "o1_pg_read"):
        go = lambda **kw: write(o1, fn=fn, **kw)
        assert go(seqs=()) == o1.O1_OK and go(rows=0, seqs=((0, 0, 1, 3),)) == o1.O1_OK
        assert go(seqs=None) == A and go(rows=-1) == A and go(seqs=((0, 0, 0, 0),) * 4097) == A
        for bad in SEQ_BAD:
            assert go(seqs=bad) == A, bad
        for name in ("k", "v"):
            assert go(**{name: None}) == A and go(**{name: MB + 8}) == A
        for name, short in (("ks", 124), ("vs", 60)):
            assert go(**{name: short}) == A and go(**{name: 1001}) == A and go(**{name: -128}) == A
        for over in (dict(k=128 * MB), dict(v=144 * MB), dict(k=162 * MB), dict(v=128 * MB)):
            assert go(**over) == A, over
        assert go(g=geom(o1, cache_dtype=E4), k=160 * MB) == A
    # a position of a slot twice: only to be read
    assert write(o1, seqs=((0, 4, 2, 0), (4, 4, 2, 3))) == A
    # outputs of a read over one another
    assert write(o1, fn="o1_pg_read", v=MB) == A


def test_chunk_refusals(o1):
    A = o1.O1_ERR_ARG
    assert chunk(o1, seqs=()) == o1.O1_OK and chunk(o1, rows=0, seqs=((0, 0, 1, 3),)) == o1.O1_OK
    assert chunk(o1, seqs=None) == A and chunk(o1, rows=-1) == A
    for bad in SEQ_BAD:
        assert chunk(o1, seqs=bad) == A, bad
    for name in ("q", "out", "scratch"):
        assert chunk(o1, **{name: None}) == A and chunk(o1, **{name: 16 * MB + 8}) == A
    assert chunk(o1, scratch=32 * MB + 16) == A
    assert chunk(o1, nbytes=o1.o1_pg_scratch_bytes(geom(o1), 8) - 1) == A
    for name, short in (("qs", 252), ("os_", 124)):
        assert chunk(o1, **{name: short}) == A and chunk(o1, **{name: 1001}) == A
    for over in (dict(out=MB), dict(out=128 * MB), dict(out=162 * MB), dict(out=32 * MB), dict(scratch=MB), dict(scratch=144 * MB),
                 dict(out=144 * MB)):
        assert chunk(o1, **over) == A, over
    assert chunk(o1, g=geom(o1, cache_dtype=E4), out=160 * MB) == A


def test_vectors_of_a_sequence(o1):
    """A sequence's rows times its heads a group are counted in 32 bits."""
    big = dict(g=geom(o1, G=1, hpg=16, d=8, dv=8, page=256), c=cache(o1, n_pages=1, width=1 << 22), q=1 << 44, qs=128, out=1 << 45,
               os_=128, rows=1 << 28)
    assert chunk(o1, seqs=((0, 1 << 27, 0, 0),), **big) == o1.O1_ERR_ARG
    assert chunk(o1, seqs=((0, 0, 0, 0), (0, 1 << 28, 1, 0)), **big) == o1.O1_ERR_ARG


def test_token_refusals(o1):
    A = o1.O1_ERR_ARG
    for call in (token, token_write):
        assert call(o1, rows=0) == o1.O1_OK
        assert call(o1, rows=-1) == A and call(o1, rows=65537) == A
        assert call(o1, pos=None) == A and call(o1, pos=7 * MB + 4) == A and call(o1, slots=6 * MB + 2) == A
        assert call(o1, slots=None, rows=5) == A       # no slots: row r uses slot r
    for name in ("q", "out", "scratch"):
        assert token(o1, **{name: None}) == A and token(o1, **{name: 16 * MB + 8}) == A
    assert token(o1, nbytes=o1.o1_pg_scratch_bytes(geom(o1), 4) - 1) == A
    for over in (dict(out=MB), dict(out=128 * MB), dict(out=6 * MB), dict(out=7 * MB), dict(scratch=6 * MB), dict(pos=32 * MB)):
        assert token(o1, **over) == A, over
    for name in ("k", "v"):
        assert token_write(o1, **{name: None}) == A and token_write(o1, **{name: MB + 8}) == A
    for over in (dict(k=128 * MB), dict(v=162 * MB), dict(slots=144 * MB), dict(pos=144 * MB)):
        assert token_write(o1, **over) == A, over


def test_binding(o1):
    with pytest.raises(OverflowError):
        o1.pg_seqs([(0, 1, 0, 2 ** 31)])
    with pytest.raises(ValueError):
        o1.pg_seqs([(0, 1, 0)])
    with pytest.raises(ValueError):
        o1.pg_geom(1, 1, 64, 64, window=2 ** 32)
    with pytest.raises(ValueError):
        o1.o1_pg_scratch_bytes(geom(o1), 2 ** 32 + 1)
    s = o1.pg_seqs([(7, 2 ** 31 - 1, 3, 9), (torch.tensor(5), 4.0, -1, 0)])
    assert [(x.row0, x.rows, x.slot, x.pos0) for x in s] == [(7, 2 ** 31 - 1, 3, 9), (5, 4, -1, 0)] and len(o1.pg_seqs([])) == 0
    g = geom(o1)
    assert g.cache_dtype == 1 and g.nh == 4 and geom(o1, dtype=HF).cache_dtype == 2
    with pytest.raises(TypeError):   # host tensors
        o1.pg_cache(g, torch.zeros(8, 2, 16, 64, dtype=BF), torch.zeros(8, 2, 16, 32, dtype=BF), torch.zeros(4, 4, dtype=torch.int32))


def test_reference_quantisation():
    """The reference's e4m3 values against torch's own conversion, and its
    exponents against their definition, at powers of two and beside them."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(500, 16, generator=gen) * torch.exp2(20 * torch.randn(500, 1, generator=gen))
    x[0], x[1, 3:] = 0.0, 0.0
    for i, top in enumerate((448.0, 449.0, 447.0, 224.0, 1.75, 1.7500001, 2.0 ** -126, 2.0 ** -149, 3.4e38)):
        x[10 + i] = 0.0
        x[10 + i, 5] = top
    y, e = ref.quantise(x)
    e = e.int() - 127
    top = x.double().abs().amax(-1)
    assert (top <= 448 * torch.exp2(e.double())).all() and (e >= -126).all()
    assert ((top > 448 * torch.exp2(e.double() - 1)) | (e == -126)).all()
    z = torch.ldexp(x.double(), -e[:, None])
    assert torch.equal(torch.ldexp(y, -e[:, None]), z.float().to(E4).double())
    x[3, 2], x[4, 0] = float("inf"), float("nan")
    y2, e2 = ref.quantise(x)
    assert torch.isnan(y2[3, 2]) and torch.isnan(y2[4, 0]) and torch.isfinite(y2).sum() == y2.numel() - 2
    assert torch.equal(y2[5:], y[5:])
