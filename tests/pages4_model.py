"""4-bit rows of the paged cache in 64 bits, from their definition.  Everything is torch on the CPU."""
import math

import torch

from tests import pages_model as pm
from video_kv_cache_gb300 import api

E2M1, INT4 = torch.float4_e2m1fn_x2, torch.uint8
TOP = {E2M1: 6.0, INT4: 7.0}
# values of the 16 codes
VALUES = {E2M1: [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
          INT4: [float(c) for c in range(8)] + [float(c - 16) for c in range(8, 16)]}
POOLS = ("k", "v", "k_scale", "v_scale", "k_group", "v_group")


def nearest(y, values):
    """Codes of the values nearest to y, halfway ones to the even code (a magnitude's last bit)."""
    v = torch.tensor(values, dtype=torch.float64)
    best = torch.full(y.shape, math.inf, dtype=torch.float64)
    code = torch.zeros(y.shape, dtype=torch.uint8)
    for c, x in enumerate(v):
        d = (y - x).abs()
        take = (d < best) | ((d == best) & (c % 2 == 0) & (code % 2 == 1))
        best, code = torch.where(take, d, best), torch.where(take, torch.tensor(c, dtype=torch.uint8), code)
    return code


def stored(x, fmt):
    """(bytes, group scales, scale) of rows x, from the definition in 64 bits."""
    x = x.double()
    g = x.unflatten(-1, (8, 16))
    ag = g.abs().amax(-1)
    a = ag.amax(-1)
    live = a >= 2.0 ** -100
    t = torch.where(live[..., None], 64 * ag / a[..., None], torch.zeros_like(ag)).float().to(torch.float8_e4m3fn)
    t64 = t.double()
    y = torch.where((t64 > 0)[..., None], g * (64 * TOP[fmt]) / (a[..., None] * t64)[..., None], torch.zeros_like(g))
    c = nearest(y.clamp(min=-7) if fmt is INT4 else y, VALUES[fmt])  # (INT4: -8 is not written)
    c = c.flatten(-2).unflatten(-1, (64, 2))
    s = torch.where(live, a / (64 * TOP[fmt]), torch.zeros_like(a)).float()
    return c[..., 0] | (c[..., 1] << 4), t, s


def decoded(raw, t, s, fmt):
    """Values of rows in 64 bits (an infinite or NaN scale times a code of 0 is NaN)."""
    v = torch.tensor(VALUES[fmt], dtype=torch.float64)
    raw = raw.view(torch.uint8)
    c = torch.stack([v[(raw & 15).long()], v[(raw >> 4).long()]], -1).flatten(-2)
    return c * t.double().repeat_interleave(16, -1) * s.double()[..., None]


def pool_rows(kv, name, table_row, n):
    """[heads][n][128] in 64 bits."""
    ids = table_row[: -(-n // kv.page_tokens)].long().cpu() if n else torch.zeros(0, dtype=torch.long)
    raw = getattr(kv, name).view(torch.uint8)[ids.to(kv.k.device)].cpu()
    t = getattr(kv, name + "_group").view(torch.uint8)[ids.to(kv.k.device)].cpu().view(torch.float8_e4m3fn)
    s = getattr(kv, name + "_scale")[ids.to(kv.k.device)].cpu()
    return decoded(raw, t, s, kv.k.dtype).transpose(0, 1).flatten(1, 2)[:, :n]


def cache(g, kv_lens, heads, fmt, page):
    """Random rows in shuffled pages; what no sequence reaches holds codes at random, NaN scales and
    NaN group scales.  Returns (pages, page table on the CPU)."""
    need = [-(-n // page) for n in kv_lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(kv_lens), max(1, max(need)) + 1), -5, dtype=torch.int32)
    written = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k].to(torch.int32)
        written[order[at:at + k]] = (torch.arange(k * page) < kv_lens[b]).view(k, page)
        at += k
    live = written[:, None, :]
    pools = {}
    for name in ("k", "v"):
        shape = (pages, heads, page)
        raw = torch.randint(0, 256, (*shape, 64), generator=g, dtype=torch.uint8)
        if fmt is INT4:  # codes of -8 are not written
            raw = torch.where(raw & 15 == 8, raw + 1, raw)
            raw = torch.where(raw >> 4 == 8, raw + 16, raw)
        t = (8 + 56 * torch.rand((*shape, 8), generator=g)).to(torch.float8_e4m3fn)
        t = torch.where(live[..., None], t.view(torch.uint8), torch.tensor(0x7F, dtype=torch.uint8))
        s = (0.2 + torch.rand(shape, generator=g)) / (32 * TOP[fmt])
        pools[name], pools[name + "_group"] = raw.view(fmt), t.view(torch.float8_e4m3fn)
        pools[name + "_scale"] = torch.where(live, s, torch.tensor(math.nan))
    return api.PagedKV(*(pools[x].cuda() for x in POOLS)), table


def seen(n, nq, window):
    """Keys [a, z) that each causal query sees."""
    pos = [n - nq + i for i in range(nq)]
    return [(max(0, p + 1 - window) if window else 0, max(0, p + 1)) for p in pos]


def attend_rows(Q, K, V, rows, spans, out_dtype, u_kv):
    """(output, lse, their bounds) of single rows over the keys that each sees and no others: fp16
    weights over 4-bit pages, everything else as pages_model.attend counts it."""
    got = [pm.attend(Q[i:i + 1], K[a:z], V[a:z], 128 ** -0.5, False, 0, pm.HALF_EPS[torch.float16], out_dtype, u_kv, u_kv)
           for i, (a, z) in ((i, spans[i]) for i in rows)]
    return tuple(torch.cat([x[k] for x in got]) for k in range(4))
