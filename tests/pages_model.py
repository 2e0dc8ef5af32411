"""The paged-cache operators in 64 bits, from their definitions, and how far fp32 arithmetic with
stated roundings may be off.  Everything is torch on the CPU."""
import math

import torch

TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
HALF_EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# smallest step of a type (half of it is the rounding of a subnormal result)
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}

# A rotated component is u c - w s times mscale.  The angle as an fp32 number of half turns is
# within 2^-24 of a half turn (1.9e-7 rad), sine and cosine within 2 ulp (2.4e-7 / 2 each at
# magnitude below 1), and two products, a sum and the factor mscale add three roundings of
# 2^-24: 1.9e-7 + 1.2e-7 + 1.8e-7 < 5.5e-7 of (|u| + |w|) mscale.
ROTATE = 5.5e-7


def rotate(X, positions, freqs, sections, interleaved, mscale=1.0, backward=False):
    """(turned X, bound on the error of the fp32 arithmetic); X [n][heads][128]."""
    X = X.double()
    half = len(freqs)
    axis = [a for a, s in enumerate(sections) for _ in range(s)]
    Y, E = X.clone(), torch.zeros_like(X)
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        ang = positions[axis[p]].double() * float(freqs[p])
        c, s = (mscale * ang.cos())[:, None], (mscale * ang.sin())[:, None]
        if backward:
            s = -s
        u, w = X[:, :, i], X[:, :, j]
        Y[:, :, i], Y[:, :, j] = u * c - w * s, u * s + w * c
        E[:, :, i] = E[:, :, j] = ROTATE * abs(mscale) * (u.abs() + w.abs())
    return Y, E


def stored(x32, dtype):
    """(codes, scale) of fp32 rows x32 in an 8-bit format, step by step in fp32 as defined."""
    top = torch.tensor(TOP[dtype], dtype=torch.float32)
    amax = x32.abs().amax(-1)
    tiny = amax < 2.0 ** -100
    r = torch.where(tiny, torch.zeros_like(amax), top / amax)
    y = x32 * r[..., None]
    codes = y.round().to(torch.int8) if dtype == torch.int8 else y.to(dtype)
    return codes, torch.where(tiny, torch.zeros_like(amax), amax / top)


def take(x, index):
    """x[index] (8-bit floats are indexed by their bytes)."""
    return x.view(torch.uint8)[index].view(x.dtype) if x.dtype in TOP else x[index]


def pool_rows(pool, scale, table_row, n, page):
    """[heads][n][128] in 64 bits."""
    ids = table_row[: -(-n // page)].long().cpu() if n else torch.zeros(0, dtype=torch.long)
    x = take(pool.cpu(), ids).double()
    if scale is not None:
        x = x * scale.cpu()[ids].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def attend(Q, K, V, scale, causal, window, u_p, out_dtype, u_k=0.0, u_v=0.0):
    """One sequence, one query head.  Q [nq][128], K and V [n][128], 64 bits.
    Returns (out, lse, bound on out's error, bound on lse's error).

    A score is 128 exact products summed in fp32 (128 roundings or truncations of at most
    2^-23 of sum |q k|), times the scale in powers of two (3 roundings): its error e_j, plus
    2^-21 for the exponential, bounds the relative error of a weight.  Weights meet the values
    rounded by u_p, or, where fp16 weights fall below its normal range, by half its smallest
    step: 2^-25 of a weight of 1 (the largest weight is at least 1, and so is their sum) times a
    value, and for 8-bit pages 2^-25 of the largest product of scale and code; keys and
    values times their scales are rounded by u_k and u_v (keys far below the largest by 2^-30 of
    it); sums over n keys add n 2^-23, a rescaling at most each 16 keys 2^-22.  The
    log-sum-exp inherits the mean e_j and 2^-21 of its own size."""
    nq, n = Q.shape[0], K.shape[0]
    pos = torch.arange(n - nq, n)[:, None]
    key = torch.arange(n)[None, :]
    seen = torch.ones(nq, n, dtype=torch.bool)
    if causal:
        seen &= key <= pos
    if window:
        seen &= key > pos - window
    s = Q @ K.T * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True) if n else torch.full((nq, 1), -math.inf, dtype=torch.float64)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    w = p / torch.where(total > 0, total, torch.ones_like(total))
    Vs = torch.where(seen.any(0)[:, None], V, torch.zeros_like(V)) if n else V
    out = w @ Vs
    lse = (m + torch.log(total))[:, 0]
    e = abs(scale) * (2.0 ** -16 + u_k) * (Q.abs() @ K.abs().T) + 2.0 ** -22 * (s.abs() + m.abs())
    if u_k and n:
        e = e + abs(scale) * 2.0 ** -30 * Q.abs().sum(-1, keepdim=True) * K.nan_to_num().abs().amax()
    e = torch.where(seen, e, torch.zeros_like(e)) + 2.0 ** -21
    mean_e = (w * e).sum(-1, keepdim=True)
    sums = n * 2.0 ** -23 + (n / 16 + 8) * 2.0 ** -22
    bound = (w * (e + (1 + u_p) * (1 + u_v) - 1 + sums)) @ Vs.abs() + out.abs() * (mean_e + sums)
    if u_p == HALF_EPS[torch.float16] and n:
        bound = bound + n * 2.0 ** -25 * Vs.abs().amax()
    bound = bound * 1.01 + out.abs() * HALF_EPS[out_dtype] + TINY[out_dtype]
    lse_bound = mean_e[:, 0] + sums + 2.0 ** -21 * (lse.abs() + 1)
    return out, lse, bound, lse_bound
