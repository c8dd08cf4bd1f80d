"""The linear layer and the head prep in 64 bits, one row at a time, on the
CPU, with the bounds their fp32 kernels are held to.

Bounds (u = 2^-24, the half step of fp32).

Linear layer. A state or output is a sum of terms k_j v_j (times q) with
weights e^{g (t - j)}. With A the same sum over absolute values:
 - a term of the row kernel goes through at most `rows` steps, each a weight
   off by 2u (expf) and a rounding: 3 u rows, rows at most ROW_STEPS where
   that kernel is taken;
 - a term of the chunk kernels carries its weights (a few u each, one a
   chunk: 8 u chunks) and is summed by at most 48 accumulations of a tensor
   core's 16-term products, each off by at most 2u of the partial sum: 128 u
   with the 16-term sums, the q products and the joins;
 - outputs of 16-bit types take the scores and the entering state in two bf16
   terms (2^-17 each).
So |error| <= (128 + 8 chunks + 3 min(rows, ROW_STEPS)) u A, + 2^-16 A for
16-bit outputs, + the output's rounding (`rounding`).

Head prep. x is exact; the sum of squares of d values is off by at most
(d/32 + 6) u, halved by the root, rsqrtf by 2 ulp (4u), the factor and the
weight by a rounding each; cosine and sine by 2 ulp (4u) and the angle's
rounding (2^-26 turn = 1.6 u rad), the products and their sum by 3 roundings:
|error| <= (24 + d/64) u (|y_j| + |y_partner|) + the output's rounding.
"""
import torch

U = 2.0 ** -24
ROW_STEPS = 64
CHUNK = 128


def rounding(z, dtype):
    """Half a step of `dtype` at z: eps/2 relative to |z|, and below the
    smallest normal number 2^-14 of fp16 (fp32 and bf16: 2^-126) the constant
    half spacing smallest_normal * eps / 2 of its subnormals."""
    f = torch.finfo(dtype)
    return (f.eps / 2) * z.abs().clamp(min=f.smallest_normal)


def linear(q, k, v, log_decay, state, seqs, scale):
    """-> out, A_out (rows of no sequence 0), state, A_state; double, CPU.
    q [R, nh, d], k [R, G, d], v [R, G, dv], state [slots, nh, d, dv]."""
    q, k, v, g = (x.detach().cpu().double() for x in (q, k, v, log_decay))
    S = state.detach().cpu().double().clone()
    nh, hpg = q.shape[1], q.shape[1] // k.shape[1]
    lam = g.exp().view(nh, 1, 1)
    out = torch.zeros(q.shape[0], nh, v.shape[2], dtype=torch.float64)
    Ao, As = torch.zeros_like(out), S.abs()
    for row0, rows, slot in seqs:
        s, a = S[slot], As[slot]
        for r in range(row0, row0 + rows):
            kk, vv = k[r].repeat_interleave(hpg, 0), v[r].repeat_interleave(hpg, 0)
            s = s * lam + kk[:, :, None] * vv[:, None, :]
            a = a * lam + (kk[:, :, None] * vv[:, None, :]).abs()
            out[r] = scale * torch.einsum("hd,hde->he", q[r], s)
            Ao[r] = abs(scale) * torch.einsum("hd,hde->he", q[r].abs(), a)
        S[slot], As[slot] = s, a
    return out, Ao, S, As


def linear_bounds(out, Ao, As, seqs, dtype):
    """Elementwise bounds of the outputs (rows of no sequence: 0) and the state."""
    bo, bs = torch.zeros_like(out), torch.zeros_like(As)
    for row0, rows, slot in seqs:
        c = (128 + 8 * -(-rows // CHUNK) + 3 * min(rows, ROW_STEPS)) * U
        r = slice(row0, row0 + rows)
        bo[r] = (c + (0 if dtype == torch.float32 else 2.0 ** -16)) * Ao[r] + rounding(out[r], dtype)
        if rows:
            bs[slot] = c * As[slot]
    return bo, bs


def prep(x, weight, inv_freq, pos, rot, norm, eps):
    """-> z, |y_j| + |y_partner| (double, CPU); pos [R] int64."""
    x = x.detach().cpu().double()
    n2 = (x * x).sum(-1, keepdim=True)
    if norm == "rms":
        n2 = n2 / x.shape[-1]
    f = torch.ones_like(n2) if norm == "none" else torch.where(n2 + eps > 0, (n2 + eps).clamp(min=1e-300) ** -0.5, 0.0)
    y = x * f
    if weight is not None:
        y = y * weight.detach().cpu().double()
    z, mag, h = y.clone(), y.abs(), rot // 2
    if rot:
        a = (pos.cpu().double()[:, None] * inv_freq.cpu().double())[:, None]
        y0, y1 = y[..., :h], y[..., h:rot]
        z[..., :h], z[..., h:rot] = y0 * a.cos() - y1 * a.sin(), y1 * a.cos() + y0 * a.sin()
        mag[..., :h] = mag[..., h:rot] = y0.abs() + y1.abs()
    return z, mag


def prep_bound(z, mag, d, dtype):
    return (24 + d / 64) * U * mag + rounding(z, dtype)


def assert_within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    err = (got - want).abs()
    beyond = err > bound
    worst = float((err / (bound + 1e-300)).max()) if err.numel() else 0.0
    print(f"{what}: worst error / bound {worst:.3f}")
    assert not beyond.any(), f"{what}: {int(beyond.sum())} values beyond the bound, worst {worst:.2f} times"
