"""The head prep and the linear layer without a GPU: sizes, and the refusals
of both entry points' C checks, which come before any CUDA call (nothing here
touches a device)."""
import ctypes

import pytest
import torch

import lin_reference as ref

V = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def o1():
    from sliding_window_landmark_gb300 import build
    build.build()
    from sliding_window_landmark_gb300 import o1 as mod
    return mod


def test_linear_sizes(o1):
    g = o1.lin_geom(2, 4, 64, 32)
    assert o1.o1_lin_state_bytes(g, 3) == 3 * 8 * 64 * 32 * 4
    assert o1.o1_lin_state_bytes(g, 0) == 0 and o1.o1_lin_scratch_bytes(g, 0, 1) == 0
    assert 0 < o1.o1_lin_scratch_bytes(g, 1, 1) <= o1.o1_lin_scratch_bytes(g, 5000, 7)
    for bad in (o1.lin_geom(0, 1, 64, 64), o1.lin_geom(1, 17, 64, 64), o1.lin_geom(1, 1, 60, 64),
                o1.lin_geom(1, 1, 64, 264), o1.lin_geom(1, 1, 64, 4), o1.lin_geom(1, 1, 64, 64, scale=float("inf"))):
        assert o1.o1_lin_state_bytes(bad, 1) == 0 and o1.o1_lin_scratch_bytes(bad, 64, 1) == 0
    bad = o1.lin_geom(1, 1, 64, 64)
    bad.dtype = 3
    assert o1.o1_lin_state_bytes(bad, 1) == 0


def _chunk(o1, g=None, state=MB, slots=4, scratch=8 * MB, nbytes=MB, q=16 * MB, qs=0, k=24 * MB, ks=0, v=32 * MB, vs=0,
           decay=48 * MB, seqs=((0, 4, 0),), out=40 * MB, os_=0, rows=8):
    g = g or o1.lin_geom(2, 2, 64, 32)
    arr = o1.lin_seqs(seqs) if seqs is not None else None
    return o1.LIB.o1_lin_chunk_attend(
        V(state), slots, ctypes.byref(g), V(scratch), nbytes, V(q), qs or 4 * 64, V(k), ks or 2 * 64, V(v), vs or 2 * 32,
        V(decay), arr, len(seqs) if seqs is not None else 1, V(out), os_ or 4 * 32, rows, None)


def test_linear_chunk_refusals(o1):
    A, U = o1.O1_ERR_ARG, o1.O1_ERR_UNSUPPORTED
    assert _chunk(o1, g=o1.lin_geom(1, 1, 12, 64)) == U
    assert _chunk(o1, seqs=()) == o1.O1_OK
    assert _chunk(o1, seqs=None) == A
    assert _chunk(o1, rows=-1) == A
    # null, misaligned, too small
    for name in ("state", "scratch", "q", "k", "v", "decay", "out"):
        assert _chunk(o1, **{name: None}) == A, name
    for name in ("state", "scratch", "q", "k", "v", "out"):
        assert _chunk(o1, **{name: 16 * MB + 8}) == A, name
    assert _chunk(o1, scratch=8 * MB + 16) == A
    assert _chunk(o1, nbytes=16) == A
    # strides: shorter than a row, not a multiple of 16 bytes, negative
    for name, short in (("qs", 4 * 64 - 4), ("ks", 2 * 64 - 4), ("vs", 2 * 32 - 4), ("os_", 4 * 32 - 4)):
        assert _chunk(o1, **{name: short}) == A, name
        assert _chunk(o1, **{name: 1001}) == A, name
        assert _chunk(o1, **{name: -1024}) == A, name
    # sequences: out of range, overlapping, a slot twice
    for bad in (((-1, 4, 0),), ((0, -1, 0),), ((0, 9, 0),), ((5, 4, 0),), ((0, 4, 4),), ((0, 4, -1),),
                ((0, 4, 0), (3, 2, 1)), ((4, 4, 0), (0, 5, 1)), ((0, 4, 2), (4, 4, 2)), ((0, 0, 1), (0, 4, 1)),
                ((2 ** 31 - 1, 2 ** 31 - 1, 0),)):
        assert _chunk(o1, seqs=bad) == A, bad
    assert _chunk(o1, slots=0) == A
    # what is written, over what is read or written
    assert _chunk(o1, out=16 * MB) == A
    assert _chunk(o1, out=MB) == A
    assert _chunk(o1, state=16 * MB) == A
    assert _chunk(o1, scratch=MB) == A
    assert _chunk(o1, scratch=16 * MB) == A
    # nothing to do
    assert _chunk(o1, rows=0, seqs=((0, 0, 1),)) == o1.O1_OK


def _token(o1, g=None, state=MB, n=4, q=16 * MB, k=24 * MB, v=32 * MB, decay=48 * MB, slots=56 * MB, out=40 * MB, rows=4):
    g = g or o1.lin_geom(2, 2, 64, 32)
    return o1.LIB.o1_lin_token_attend(V(state), n, ctypes.byref(g), V(q), 256, V(k), 128, V(v), 64, V(decay), V(slots),
                                      V(out), 128, rows, None)


def test_linear_token_refusals(o1):
    A = o1.O1_ERR_ARG
    assert _token(o1, rows=0) == o1.O1_OK
    assert _token(o1, rows=-1) == A
    assert _token(o1, rows=65537) == A
    assert _token(o1, g=o1.lin_geom(1, 1, 64, 60)) == o1.O1_ERR_UNSUPPORTED
    for name in ("state", "q", "k", "v", "decay", "out"):
        assert _token(o1, **{name: None}) == A, name
    assert _token(o1, slots=56 * MB + 2) == A
    assert _token(o1, slots=None, rows=5) == A       # no slots: row r uses slot r
    assert _token(o1, out=16 * MB) == A and _token(o1, slots=40 * MB) == A and _token(o1, slots=MB) == A


def _prep(o1, g=None, q=MB, qs=256, k=2 * MB, ks=128, wq=8 * MB, wk=9 * MB, inv=10 * MB, pos=11 * MB, rows=4, qo=4 * MB,
          qos=256, ko=6 * MB, kos=128):
    g = g or o1.prep_geom(4, 2, 64)
    return o1.LIB.o1_head_prep(ctypes.byref(g), V(q), qs, V(k), ks, V(wq), V(wk), V(inv), V(pos), 0, rows, V(qo), qos,
                               V(ko), kos, None)


def test_prep_refusals(o1):
    A, U = o1.O1_ERR_ARG, o1.O1_ERR_UNSUPPORTED
    bf, hf = torch.bfloat16, torch.float16
    for bad in (o1.prep_geom(0, 0, 64), o1.prep_geom(4, 2, 60), o1.prep_geom(4, 2, 264), o1.prep_geom(4, 2, 64, rot=4),
                o1.prep_geom(4, 2, 64, rot=72), o1.prep_geom(4, 2, 64, eps=-1.0), o1.prep_geom(4, 2, 64, eps=float("nan")),
                o1.prep_geom(4, 2, 64, in_dtype=bf, out_dtype=hf), o1.prep_geom(-1, 2, 64),
                o1.prep_geom(4, 2, 64, in_dtype=torch.float32, out_dtype=bf)):
        assert _prep(o1, g=bad) == U
    assert _prep(o1, rows=0) == o1.O1_OK
    assert _prep(o1, rows=-1) == A
    for name in ("q", "k", "qo", "ko", "inv"):
        assert _prep(o1, **{name: None}) == A, name
    for name in ("q", "k", "qo", "ko", "wq", "wk"):
        assert _prep(o1, **{name: 16 * MB + 8}) == A, name
    assert _prep(o1, pos=11 * MB + 4) == A
    for name, short in (("qs", 252), ("ks", 124), ("qos", 252), ("kos", 124)):
        assert _prep(o1, **{name: short}) == A and _prep(o1, **{name: 1001}) == A
    # outputs over another tensor; over an input of another type or stride
    assert _prep(o1, ko=MB) == A and _prep(o1, qo=2 * MB) == A and _prep(o1, qo=8 * MB) == A
    assert _prep(o1, qo=10 * MB) == A and _prep(o1, qo=11 * MB) == A and _prep(o1, ko=4 * MB) == A
    assert _prep(o1, qo=MB, qos=512) == A
    mixed = o1.prep_geom(4, 2, 64, in_dtype=bf, out_dtype=torch.float32)
    assert _prep(o1, g=mixed, qo=MB) == A
    # interleaved columns that do meet: k starts inside q's columns
    assert _prep(o1, q=MB, qs=512, k=MB + 4 * 128, ks=512, qo=MB, qos=512) == A


def test_reference_state_is_the_closed_form():
    """The 64-bit reference against the sum it stands for (no recurrence)."""
    gen = torch.Generator().manual_seed(1)
    rows, nh, G, d, dv = 9, 4, 2, 8, 8
    q, k, v = (torch.randn(rows, h, w, generator=gen) for h, w in ((nh, d), (G, d), (G, dv)))
    g = -torch.rand(nh, generator=gen)
    S0 = torch.randn(2, nh, d, dv, generator=gen)
    out, Ao, S, As = ref.linear(q, k, v, g, S0, [(2, 6, 1)], 0.5)
    for h in range(nh):
        for t in range(6):
            lam = g[h].double().exp()
            want = lam ** (t + 1) * S0[1, h].double()
            for j in range(t + 1):
                want = want + lam ** (t - j) * torch.outer(k[2 + j, h // 2], v[2 + j, h // 2]).double()
            torch.testing.assert_close(out[2 + t, h], 0.5 * q[2 + t, h].double() @ want, rtol=1e-6, atol=1e-6)
        torch.testing.assert_close(S[1, h], want, rtol=1e-6, atol=1e-6)
    assert (out[:2] == 0).all() and (out[8:] == 0).all() and torch.equal(S[0], S0[0].double())
    assert (Ao >= out.abs()).all() and (As >= S.abs() - 1e-12).all()


def test_binding_counts_past_32_bits(o1):
    """Refused, where ctypes would take them modulo 2^32."""
    g = o1.lin_geom(2, 2, 64, 64)
    for bad in ((2 ** 32, 4, 0), (0, 2 ** 32 + 4, 0), (0, 4, 2 ** 32), (0, 4, -2 ** 31 - 1)):
        with pytest.raises(OverflowError):
            o1.lin_seqs([(0, 4, 1), bad])
    with pytest.raises(ValueError):
        o1.lin_seqs([(0, 4)])
    for call in (lambda n: o1.o1_lin_state_bytes(g, n), lambda n: o1.o1_lin_scratch_bytes(g, n),
                 lambda n: o1.o1_lin_scratch_bytes(g, 5, n)):
        with pytest.raises(ValueError):
            call(2 ** 32 + 1)
    s = o1.lin_seqs([(7, 2 ** 31 - 1, 3), (torch.tensor(5), 4.0, -1)])
    assert [(x.row0, x.rows, x.slot) for x in s] == [(7, 2 ** 31 - 1, 3), (5, 4, -1)] and len(o1.lin_seqs([])) == 0


def test_sizes_past_64_bits(o1):
    """The largest states: their bytes, or 0 where 64 bits do not hold them; a
    scratch for any counts is no smaller than one for fewer."""
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        big = o1.lin_geom(4095, 16, 256, 256, dtype=dt)
        one = 4095 * 16 * 256 * 256 * 4
        most = (2 ** 64 - 1) // one
        assert o1.o1_lin_state_bytes(big, most) == most * one
        for n in (most + 1, 2 ** 30 + 2 ** 20, 2 ** 31 - 1):
            assert n > most and o1.o1_lin_state_bytes(big, n) == 0
        for g in (big, o1.lin_geom(2, 2, 64, 64, dtype=dt), o1.lin_geom(1, 1, 8, 8, dtype=dt)):
            sizes = [o1.o1_lin_scratch_bytes(g, r, n) for r, n in
                     ((1, 1), (4096, 1), (2 ** 20, 4096), (2 ** 31 - 1, 2 ** 24), (2 ** 31 - 1, 2 ** 30), (2 ** 31 - 1, 2 ** 31 - 1))]
            assert 0 < sizes[0] and sizes == sorted(sizes), sizes
