"""o1_head_prep on the GPU against the 64-bit reference, held to the bounds
derived in lin_reference: norms, rotation widths, element types, widths,
strides, in place, far positions, and its result feeding a sealed layer."""
from fractions import Fraction

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


def freqs(rot, base=1e6):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()


# rows, q heads, k heads, d, rot, norm, in, out, weights
CASES = [
    (1, 8, 2, 256, 256, "rms", F32, F32, True), (1, 1, 0, 8, 8, "unit", F32, F32, False),
    (5, 0, 3, 64, 64, "unit", BF16, BF16, True), (37, 3, 1, 72, 24, "rms", F16, F32, True),
    (64, 4, 4, 128, 0, "rms", BF16, F32, False), (130, 2, 1, 200, 56, "none", F16, F16, True),
    (3, 16, 4, 128, 128, "rms", BF16, BF16, True), (33, 5, 2, 248, 248, "unit", F32, F32, True),
    (7, 2, 2, 32, 16, "none", F32, F32, False), (1001, 9, 3, 256, 64, "rms", F16, F16, True),
    (4099, 1, 1, 136, 136, "unit", BF16, F32, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("positions", ["given", "counted"])
def test_prep(o1, case, positions):
    rows, hq, hk, d, rot, norm, tin, tout, weights = CASES[case]
    gen = torch.Generator().manual_seed(case)
    q, k = (torch.randn(rows, h, d, generator=gen).mul(3).to(tin).cuda() for h in (hq, hk))
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=gen)).cuda() if weights else None for _ in range(2))
    inv = freqs(rot).cuda()
    pos0 = 12345
    pos = torch.randint(0, 1 << 22, (rows,), generator=gen).cuda() if positions == "given" else None
    g = o1.prep_geom(hq, hk, d, rot=rot, norm=norm, in_dtype=tin, out_dtype=tout, eps=1e-5)
    qo, ko = (torch.full((rows, h, d), float("nan"), dtype=tout, device="cuda") for h in (hq, hk))
    o1.check(o1.o1_head_prep(g, q if hq else None, k if hk else None, wq, wk, inv if rot else None, qo if hq else None,
                             ko if hk else None, pos=pos, pos0=pos0) if hq else
             o1.o1_head_prep(g, None, k, None, wk, inv, None, ko, pos=pos, pos0=pos0))
    torch.cuda.synchronize()
    p = pos if pos is not None else torch.arange(pos0, pos0 + rows)
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        z, mag = ref.prep(x, w, inv, p, rot, norm, g.eps)
        ref.assert_within(got, z, ref.prep_bound(z, mag, d, tout), f"case {case}")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_in_place_in_fused_rows(o1, dt):
    """q and k normalised and rotated where they lie in a projection's rows; the value columns stay."""
    rows, hq, hk, d = 50, 4, 2, 128
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(rows, (hq + 2 * hk) * d, generator=gen).to(dt).cuda()
    before = x.clone()
    view = lambda t: (t[:, :hq * d].unflatten(1, (hq, d)), t[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)))
    q, k = view(x)
    inv = freqs(d).cuda()
    g = o1.prep_geom(hq, hk, d, in_dtype=dt, eps=1e-6)
    o1.check(o1.o1_head_prep(g, q, k, None, None, inv, q, k, pos0=7))
    torch.cuda.synchronize()
    for src, got in zip(view(before), (q, k)):
        z, mag = ref.prep(src, None, inv, torch.arange(7, 7 + rows), d, "rms", g.eps)
        ref.assert_within(got, z, ref.prep_bound(z, mag, d, dt), "in place")
    assert torch.equal(x[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_zero_heads_and_no_epsilon(o1):
    q = torch.zeros(2, 2, 64, device="cuda")
    q[1, 1] = 1e-3
    out = torch.full_like(q, float("nan"))
    for norm in ("rms", "unit"):
        g = o1.prep_geom(2, 0, 64, norm=norm, eps=0.0)
        o1.check(o1.o1_head_prep(g, q, None, None, None, freqs(64).cuda(), out, None))
        torch.cuda.synchronize()
        assert (out[0] == 0).all() and (out[1, 0] == 0).all()
        z, mag = ref.prep(q, None, freqs(64), torch.arange(2), 64, norm, 0.0)
        ref.assert_within(out, z, ref.prep_bound(z, mag, 64, F32), norm)


# pi to 40 decimals
PI = Fraction(31415926535897932384626433832795028841971, 10 ** 40)


@pytest.mark.parametrize("p", [0, 1, (1 << 31) - 1, (1 << 31) + 5, 1 << 40, 123456789012])
def test_far_positions(o1, p):
    """Angles of positions past 32 bits: the exact rational angle modulo 2 pi."""
    d = 64
    inv = freqs(d)
    inv[1], inv[2], inv[3], inv[4] = 1e-30, 0.0, 3.0, 4097.5
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(1, 3, d, generator=gen).cuda()
    out = torch.empty_like(q)
    g = o1.prep_geom(3, 0, d, norm="none")
    o1.check(o1.o1_head_prep(g, q, None, None, None, inv.cuda(), out, None, pos=torch.tensor([p], device="cuda")))
    torch.cuda.synchronize()
    turns = [Fraction(float(f)) * p / (2 * PI) for f in inv.tolist()]
    ang = torch.tensor([float((t - int(t)) * 2 * PI) for t in turns], dtype=torch.float64)
    z, mag = ref.prep(q, None, ang.float(), torch.ones(1, dtype=torch.int64), d, "none", 0.0)   # shapes and mag only
    x = q.cpu().double()
    x0, x1 = x[..., :d // 2], x[..., d // 2:]
    z[..., :d // 2], z[..., d // 2:] = x0 * ang.cos() - x1 * ang.sin(), x1 * ang.cos() + x0 * ang.sin()
    # the angle's truncation: p 2^-64 turns
    ref.assert_within(out, z, ref.prep_bound(z, mag, d, F32) + mag * abs(p) * 2.0 ** -64 * 6.3, f"position {p}")


def test_captured_and_on_another_stream(o1):
    rows, d = 9, 128
    q, pos = torch.randn(rows, 4, d, device="cuda"), torch.arange(rows, device="cuda")
    out, inv = torch.empty_like(q), freqs(d).cuda()
    g = o1.prep_geom(4, 0, d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o1.check(o1.o1_head_prep(g, q, None, None, None, inv, out, None, pos=pos, stream=st))
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o1.check(o1.o1_head_prep(g, q, None, None, None, inv, out, None, pos=pos))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    pos.add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    z, mag = ref.prep(q, None, inv, pos, d, "rms", 1e-6)
    ref.assert_within(out, z, ref.prep_bound(z, mag, d, F32), "replay")


def test_binding_refuses_wrong_tensors(o1):
    q, out, inv = torch.randn(3, 2, 64, device="cuda"), torch.empty(3, 2, 64, device="cuda"), freqs(64).cuda()
    g = o1.prep_geom(2, 0, 64)
    for bad, err in (((q.half(), out), TypeError), ((q, out.cpu()), TypeError), ((q[:2], out), ValueError),
                     ((q.flip(0)[:, :, ::2], out), ValueError)):
        with pytest.raises(err):
            o1.o1_head_prep(g, bad[0], None, None, None, inv, bad[1], None)
    with pytest.raises(ValueError):
        o1.o1_head_prep(g, q, None, None, None, inv[:5], out, None)
    assert o1.o1_head_prep(g, q, None, None, None, None, out, None) == o1.O1_ERR_ARG


def test_prepared_rows_feed_a_sealed_layer(o1):
    """Norm and rotation here, then a sealed layer without a rotation of its
    own: the layer's outputs on normalised rows that it rotates itself."""
    import harness
    from sliding_window_landmark_gb300 import synth
    sh = synth.Shape(groups=2, heads_per_group=2, d=64, dv=64, sinks=2, window=48, landmarks=4)
    flat = synth.Shape(groups=2, heads_per_group=2, d=64, dv=64, sinks=2, window=48, landmarks=4, rope_base=0.0)
    c = synth.layer_constants(sh, 9)
    q, k, v, gate = synth.layer_rows(sh, 9, 0, 130)
    tq, tk = torch.from_numpy(q).cuda(), torch.from_numpy(k).cuda()
    qo, ko = torch.empty_like(tq), torch.empty_like(tk)
    g = o1.prep_geom(sh.nh, sh.groups, 64)
    o1.check(o1.o1_head_prep(g, tq, tk, None, None, freqs(64, sh.rope_base).cuda(), qo, ko))
    torch.cuda.synchronize()
    nq, nk = ((x / (x * x + 0.0).mean(-1, keepdims=True) ** 0.5) for x in (q.astype("f8"), k.astype("f8")))
    orc = harness.oracle_layer(sh, c)
    want, diag = orc.rows(nq.astype("f4"), nk.astype("f4"), v, gate, diag=True)
    got = harness.GpuLayer(flat, c, max_rows=130).rows(qo.cpu().numpy(), ko.cpu().numpy(), v, gate)
    harness.assert_outputs(got, want, diag, "prepared rows")


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("norm", ["rms", "unit"])
@pytest.mark.parametrize("d,rot", [(72, 24), (256, 256), (16, 0)])
def test_a_nan_spoils_its_whole_head(o1, dt, norm, d, rot):
    """A norm with a NaN in it is NaN: every value of that head, and no other head's."""
    gen = torch.Generator().manual_seed(13)
    q, k = (torch.randn(6, h, d, generator=gen).to(dt) for h in (3, 2))
    q[1, 2, 5] = k[3, 0, d - 1] = float("nan")
    q[5, 0] = float("nan")
    inv, pos = freqs(rot), torch.arange(100, 106)
    qo, ko = torch.zeros(6, 3, d, dtype=dt, device="cuda"), torch.zeros(6, 2, d, dtype=dt, device="cuda")
    g = o1.prep_geom(3, 2, d, rot=rot, norm=norm, in_dtype=dt)
    o1.check(o1.o1_head_prep(g, q.cuda(), k.cuda(), None, None, inv.cuda() if rot else None, qo, ko, pos0=100))
    torch.cuda.synchronize()
    for x, got in ((q, qo.cpu()), (k, ko.cpu())):
        bad = torch.isnan(x).any(-1)
        assert torch.isnan(got[bad]).all()
        z, mag = ref.prep(x, None, inv, pos, rot, norm, g.eps)
        ref.assert_within(got[~bad], z[~bad], ref.prep_bound(z, mag, d, dt)[~bad], "other heads")


# 2^-149 is the smallest fp32 value: heads of one or two steps of it too
@pytest.mark.parametrize("size", [1e-13, 1e-19, 1e-22, 1e-30, 1e-38, 2.0 ** -148])
@pytest.mark.parametrize("eps", [0.0, 1e-37, 1e-44])
@pytest.mark.parametrize("norm,d,rot", [("unit", 64, 64), ("rms", 256, 128), ("rms", 200, 56), ("unit", 8, 0)])
def test_tiny_heads_with_little_or_no_epsilon(o1, size, eps, norm, d, rot):
    """Heads whose squares leave fp32's range, beside heads of common size and zero heads."""
    gen = torch.Generator().manual_seed(17)
    q = torch.randn(5, 7, d, generator=gen)
    q[1:] *= size
    q[2, 3], q[3] = 0.0, q[0] * 1e3
    inv = freqs(rot)
    g = o1.prep_geom(7, 0, d, rot=rot, norm=norm, eps=eps)
    out = torch.full((5, 7, d), float("nan"), device="cuda")
    o1.check(o1.o1_head_prep(g, q.cuda(), None, None, None, inv.cuda() if rot else None, out, None, pos0=3))
    torch.cuda.synchronize()
    z, mag = ref.prep(q, None, inv, torch.arange(3, 8), rot, norm, g.eps)
    ref.assert_within(out, z, ref.prep_bound(z, mag, d, F32), f"{norm} of {size} with {eps}")


def test_more_rows_than_a_call_counts(o1):
    """A row count past 32 bits is refused, not taken modulo 2^32."""
    g = o1.prep_geom(1, 0, 8, rot=0)
    q = torch.zeros(1, 1, 8, device="cuda").expand(2 ** 32 + 5, 1, 8)
    with pytest.raises(ValueError):
        o1.o1_head_prep(g, q, None, None, None, None, q, None)
