"""The paged cache and the attention over it in 64 bits, with the bounds their
kernels are held to.

Cache. Rounding to bf16 or fp16 is torch's (nearest, ties to even). e4m3: for a
head's row x, 2^e is the least power of two, e >= -126, with max |x| <= 448 2^e
over its finite values; x / 2^e is rounded to the nearest multiple of
2^(max(floor(log2 |x / 2^e|), -6) - 3), ties to even, in 64 bits, where nothing
else rounds. What the cache holds must be these values exactly.

Attention (u = 2^-24, the half step of fp32). Over a row's attended positions,
w_j = e^{s_j}, s_j = scale q.k_j, S_j = |scale| sum |q| |k_j|, p_j = w_j / sum w.
 - A score is a sum of d products on the tensor cores, TERMS terms of q each in
   steps of 16, each accumulation off by at most 2u of what is summed, and is
   scaled and taken from a reference r in log2 units (4 roundings of |s_j| or
   |s_j - r|, and |r| is some |s_i| of the row): with M = max |s_i|,
   (2 (d / 16 + 2) TERMS u) S_j + 8 u M; terms of q hold it to
   2^-24 of S_j at least, counted as 2u. ex2.approx is off by 2^-22.
   delta_j, their sum, is the relative error of w_j.
 - The weights of the values are rounded to rho: bf16 has 8 significant bits, so
   a value in [1, 2) is off by at most half of 2^-7: 2^-8 relative for one bf16
   term, 2^-16 for two (the second takes what the first left, at most 2^-8, and
   leaves 2^-8 of it), 2^-24 for three; fp16, 11 bits, 2^-11, and 2^-25 below its
   normal numbers. fp16 weights of an e4m3 cache are those of the codes v_j /
   2^{e_j}, that is p_j 2^{e_j}, and are taken so that a row's largest is at least
   1: 2^-25 max_i (p_i 2^{e_i}) sum_j |v_j| / 2^{e_j} (e = 0 for an fp16 cache).
 - 16-bit rows over e4m3: q in fp16 times a power of two that brings its largest
   value into [1, 2): 2^-25 of that value for each of q's below 2^-14, so 2^-25
   |scale| max |q| sum |k_j| of a score.
 - The weighted sum is n / 8 + 400 accumulations or joins, n the keys, each off
   by at most 2u of the absolute sum.
So with A = sum p_j |v_j|: |error| <= sum p_j delta_j (|v_j| + |out|)
 + (rho + (n / 4 + 800) u) A + the output's rounding, doubled for products of
these errors where they are not small (they are all below 2^-7 here: 1.01).
"""
import torch

from lin_reference import U, assert_within, rounding  # noqa: F401

E4M3 = torch.float8_e4m3fn


def pow2(e):
    """2^e as a double, from its bits: pow and exp2 are not exact on every device."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantise(x):
    """-> values x is held as (double), and the byte e + 127 of each row."""
    x = x.double()
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1, keepdim=True)
    m, e = torch.frexp(top)                                     # top = m 2^e, m in [1/2, 1)
    e = torch.where(top > 0, e - 8 - (m <= 0.875).to(e.dtype), -126).clamp(min=-126)   # 448 = 0.875 2^9
    y = x * pow2(-e)
    step = pow2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)   # frexp's exponent is floor(log2) + 1
    y = torch.where(torch.isfinite(x), torch.round(y / step) * step, float("nan"))
    return y * pow2(e), (e + 127)[..., 0].to(torch.uint8)


def held(pool, exp):
    """The values a pool holds, double."""
    x = pool.double()
    return x if exp is None else x * pow2(exp.int()[..., None] - 127)


def places(table, page, slot, a, b):
    """Page and row in it of positions a .. b - 1."""
    p = torch.arange(a, b, device=table.device)
    return table[slot, p // page].long(), p % page


def attend(q, k, v, table, page, n_pages, seqs, scale, window, dtype, terms, rho, f16_weights=False, v_exp=None):
    """-> out and its bound (double; rows of no sequence 0). k, v: held values
    [pages, G, page, width]; seqs (row0, rows, slot, pos0); v_exp: the values'
    bytes of an e4m3 cache."""
    q = q.double()
    R, nh, d = q.shape
    G, dv = k.shape[1], v.shape[3]
    out = torch.zeros(R, nh, dv, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for row0, rows, slot, pos0 in seqs:
        if rows == 0:
            continue
        p = torch.arange(pos0, pos0 + rows, device=q.device)
        a = max(0, pos0 - window + 1) if window else 0
        ids, at = places(table, page, slot, a, pos0 + rows)
        there = (ids >= 0) & (ids < n_pages)
        ids = torch.where(there, ids, 0)
        j = torch.arange(a, pos0 + rows, device=q.device)
        see = (j <= p[:, None]) & there
        if window:
            see &= j > p[:, None] - window
        kk, vv = k[ids, :, at].transpose(0, 1), v[ids, :, at].transpose(0, 1)          # [G, n, width]
        qq = q[row0:row0 + rows].unflatten(1, (G, nh // G)).permute(1, 2, 0, 3)        # [G, hpg, rows, d]
        s = scale * (qq @ kk[:, None].transpose(-1, -2))
        S = abs(scale) * (qq.abs() @ kk[:, None].abs().transpose(-1, -2))
        s, S = torch.where(see, s, -float("inf")), torch.where(see, S, 0.0)
        top = torch.where(see, s.abs(), 0.0).amax(-1, keepdim=True)
        big = s.amax(-1, keepdim=True)
        w = torch.exp(s - torch.where(big > -float("inf"), big, 0.0))
        l = w.sum(-1, keepdim=True)
        pr = w / torch.where(l > 0, l, 1.0)
        o = pr @ vv[:, None]
        A = pr @ vv[:, None].abs()
        delta = (2 * (d / 16 + 2) * terms + 2) * U * S + 8 * U * top + 2.0 ** -22
        if v_exp is not None and dtype is not torch.float32:
            far = abs(scale) * qq.abs().amax(-1, keepdim=True) * kk[:, None].abs().sum(-1)[..., None, :]
            delta = delta + 2.0 ** -25 * torch.where(see, far, 0.0)
        b = 1.01 * ((pr * delta) @ vv[:, None].abs() + (pr * delta).sum(-1, keepdim=True) * o.abs()
                    + (rho + (j.numel() / 4 + 800) * U) * A)
        if f16_weights:
            size = pow2(v_exp[ids, :, at].int() - 127).T if v_exp is not None else torch.ones_like(vv[..., 0])   # [G, n]
            most = (pr * size[:, None, None]).amax(-1, keepdim=True)
            b = b + 2.0 ** -25 * most * (see.double() @ (vv.abs() / size[..., None])[:, None])
        out[row0:row0 + rows] = o.permute(2, 0, 1, 3).flatten(1, 2)
        bound[row0:row0 + rows] = b.permute(2, 0, 1, 3).flatten(1, 2)
    return out, bound + rounding(out, dtype)


def precision(dtype, cache_dtype):
    """Terms, rho and whether weights are fp16, of rows over a cache."""
    if dtype is torch.float32:
        return 3, 2.0 ** -24, False
    if cache_dtype is E4M3:   # in fp16 or, for many rows, in bf16
        return 2, 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -11, True
    return (1, 2.0 ** -8, False) if dtype is torch.bfloat16 else (1, 2.0 ** -11, True)
