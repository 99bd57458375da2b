"""float64 references and derived tolerances of the device-planned serving
operators (plain tensor arithmetic on CPU; no code of the CUDA path)."""

from __future__ import annotations

import math

import torch

# A rounding to bf16, f16 or E4M3 is off by at most half a step.
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_F16 = torch.finfo(torch.float16).eps / 2
HALF_E4M3 = 2.0 ** -4


def rotate(x, pos, cos_sin, rot_start, interleaved):
    """x [T, heads, d] at positions pos, turned by rows of cos_sin; float64."""
    y = x.double().clone()
    if cos_sin is None:
        return y
    r = cos_sin.shape[1]
    c, s = cos_sin.double()[pos][:, None, :].chunk(2, dim=-1)
    mid = y[..., rot_start:rot_start + r]
    if interleaved:
        a, b = mid[..., 0::2].clone(), mid[..., 1::2].clone()
        mid[..., 0::2], mid[..., 1::2] = a * c - b * s, b * c + a * s
    else:
        a, b = mid[..., : r // 2].clone(), mid[..., r // 2:].clone()
        mid[..., : r // 2], mid[..., r // 2:] = a * c - b * s, b * c + a * s
    return y


def rotate_slack(x, cos_sin):
    """Error of the float32 products and their sum: two products and one sum,
    each rounded (2^-24), of magnitudes at most |x| + |y| <= 2 max|x| (cos and
    sin are at most 1)."""
    return 0.0 if cos_sin is None else 3 * 2.0 ** -24 * 2 * float(x.double().abs().max())


def attend(q, k, v, scale, causal):
    """softmax(q k^T scale) v of one sequence: q [n, H, dq], k [m, Hkv, dq],
    v [m, Hkv, dv] (n = m when causal); returns out [n, H, dv], lse [H, n],
    and sum_j w_j |v_j| and max_j sum_i |q_i k_i| scale, which the tolerances use."""
    n, H, dq = q.shape
    m, Hkv, dv = v.shape
    g = H // Hkv
    qq = q.double().view(n, Hkv, g, dq)
    kk, vv = k.double(), v.double()
    s = torch.einsum("nhgd,mhd->hgnm", qq, kk) * scale
    mag = torch.einsum("nhgd,mhd->hgnm", qq.abs(), kk.abs()) * scale
    if causal:
        hide = torch.ones((n, m), dtype=torch.bool).triu(1)
        s = s.masked_fill(hide, -math.inf)
        mag = mag.masked_fill(hide, 0.0)
    lse = torch.logsumexp(s, -1)
    w = (s - lse[..., None]).exp()
    out = torch.einsum("hgnm,mhd->nhgd", w, vv).reshape(n, H, dv)
    absw = torch.einsum("hgnm,mhd->nhgd", w, vv.abs()).reshape(n, H, dv)
    return out, lse.reshape(H, n), absw, mag.amax(-1).reshape(H, n)


def check_attention(out, lse, ref, dq, half_p, what=""):
    """out [n, H, dv] and lse [H, n] against attend()'s tuple.

    A score is a sum of dq exact products accumulated in float32 in any order,
    each addition off by at most 2^-23 of the running magnitude (truncating
    adders included), so |ds| <= dq 2^-23 sum|q_i k_i| scale, and the exponent
    2^x of its float32 argument adds 2^-22 |s| + 2^-21.  A weight is then off by
    2 ds' relative (numerator and denominator), its rounding for the product
    with v by half_p, the sums over keys by 2^-16 (chains of at most 2^7 adds
    between rescales and joins); the result is rounded to bf16 once."""
    o, l, absw, mag = ref
    ds = mag * dq * 2.0 ** -23 + mag * 2.0 ** -22 + 2.0 ** -21
    err = (out.double().cpu() - o).abs()
    tol = HALF_BF16 * o.abs() + (half_p + 2 * ds.t()[..., None] + 2.0 ** -16) * absw * (1 + HALF_BF16) + 1e-30
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert torch.isfinite(out.float()).all(), f"{what}: non-finite output"
    assert worst <= 1.0, f"{what}: output off by {worst:.3f} of its tolerance"
    if lse is not None:
        lerr = (lse.double().cpu() - l).abs()
        ltol = ds + 2.0 ** -16 + 2.0 ** -22 * l.abs()
        lworst = float((lerr / ltol).max()) if lerr.numel() else 0.0
        assert lworst <= 1.0, f"{what}: lse off by {lworst:.3f} of its tolerance"
    return worst


def randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def block_table(ctx, seed, spare=2):
    """A table over a shuffled pool (-1 where unused) and the pool's size."""
    pages = [-(-n // 64) for n in ctx]
    pool = sum(pages) + spare
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(ctx), max(1, max(pages, default=1))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table, pool


def fill_cache(cache, table, b, rows):
    """Writes rows [n, kv_heads, d] to positions 0 .. n-1 of sequence b (CPU)."""
    n = rows.shape[0]
    pos = torch.arange(n)
    cache[table[b].long()[pos // 64], pos % 64] = rows
