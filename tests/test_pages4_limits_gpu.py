"""GPU checks of 4-bit pages at the ends of their ranges: weights and value scales as large as the running
references let them get, every group scale read back, keys of any bits that a mask hides."""
import math

import numpy as np
import pytest
import torch

from tests import pages4_model as m4
from tests import pages_model as pm
from tests import test_pages_gpu as tp
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu
BF, HF, F32, E2M1, INT4 = torch.bfloat16, torch.float16, torch.float32, m4.E2M1, m4.INT4
JUST_BELOW_8 = float(np.nextafter(np.float32(8), np.float32(0)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


def _one_key_above(fmt, n, at, base, above, size):
    """n keys of score `base` and value 1, but for key `at`: score base + above, value `size`."""
    page = 64
    kv = api.allocate_pages(-(-n // page), 1, page, fmt)
    code = {v: c for c, v in enumerate(m4.VALUES[fmt])}
    kv.k.view(torch.uint8).zero_()
    kv.k.view(torch.uint8)[..., 0] = code[4.0]                # channel 0 of the keys alone
    kv.k_group.view(torch.uint8).fill_(0x40)                  # 2
    kv.k_scale.fill_(base / 8)
    kv.v.view(torch.uint8).fill_(code[1.0] * 17)
    kv.v_group.view(torch.uint8).fill_(0x38)                  # 1
    kv.v_scale.fill_(1.0)
    kv.k_scale[at // page, 0, at % page] = (base + above) / 8
    kv.v_scale[at // page, 0, at % page] = size
    return kv, torch.arange(kv.n_pages, dtype=torch.int32).view(1, -1)


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("n", [256, 2048])        # one item, and four splits of it
@pytest.mark.parametrize("base,above,size", [
    (0.0, 7.9999, JUST_BELOW_8),                  # neither the base of the weights nor the values' reference moves
    (0.0, 7.9999, -JUST_BELOW_8),
    (0.0, 7.999, 7.9),
    (2.0 ** 20, 8.0, 7.0),
    (2.0 ** 22, 7.5, JUST_BELOW_8),
    (2.0 ** 23 - 16, 8.0, 7.0),
])
def test_a_weight_and_a_value_scale_at_their_limits(fmt, n, base, above, size):
    # key 200 lies in the second tile, which goes by the first one's references: its weight may be 2^8, and
    # its value's scale eight times the first tile's.  Weights meet the values in fp16
    nq, at = 40, 200
    kv, table = _one_key_above(fmt, n, at, base, above, size)
    Q = torch.zeros((nq, 1, 128), dtype=HF)
    Q[:, :, 0] = 1.0
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    K, V = m4.pool_rows(kv, "k", table[0], n)[0], m4.pool_rows(kv, "v", table[0], n)[0]
    for causal in (False, True):
        for out_dtype, lse in ((F32, False), (HF, True), (BF, True)):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = api.page_attention(Q.cuda(), kv, table.cuda(), lens, causal=causal, scale=math.log(2), out_dtype=out_dtype,
                                     return_lse=lse, status=status)
            want, want_lse, bound, lse_bound = pm.attend(Q[:, 0].double(), K, V, math.log(2), causal, 0, 2.0 ** -11, out_dtype)
            if lse:
                tp._within(got[1][:, 0], want_lse, lse_bound, "lse")
                got = got[0]
            assert int(status) == 0
            tp._within(got[:, 0], want, bound, "output")


@pytest.mark.parametrize("fmt", [E2M1, INT4])
def test_reads_give_what_every_group_scale_stands_for(fmt):
    # all 256 bytes, over 64 (which page_write does not store) and NaN among them, with all 16 codes each: a
    # scale times a code is exact, and one rounding is left, that of the row's scale
    kv = api.allocate_pages(2, 1, 16, fmt)
    codes = torch.tensor([(2 * i) | (2 * i + 1) << 4 for i in range(8)], dtype=torch.uint8).repeat(8)
    scales = torch.arange(256).to(torch.uint8).view(2, 1, 16, 8)
    for pool, group in ((kv.k, kv.k_group), (kv.v, kv.v_group)):
        pool.view(torch.uint8).copy_(codes.expand(2, 1, 16, 64))
        group.view(torch.uint8).copy_(scales)
    table, lens = torch.tensor([[0, 1]], dtype=torch.int32), torch.tensor([32], dtype=torch.int32).cuda()
    for ks, vs in ((1.0, 0.3), (0.0, -2.0 ** 100)):
        kv.k_scale.fill_(ks)
        kv.v_scale.fill_(vs)
        X = api.page_read(kv, table.cuda(), lens, 32, out_dtype=F32)[0].cpu()
        for which, name in enumerate(("k", "v")):
            want = m4.pool_rows(kv, name, table[0], 32)[0].float()
            assert torch.equal(X[which].isnan(), want.isnan()) and int(want.isnan().sum()) == 32
            assert torch.equal(X[which].nan_to_num(), want.nan_to_num())


SPANS = [  # queries, cached tokens, query heads, window, a key that only some queries see
    (5, 300, 2, 0, 297), (7, 900, 2, 300, 596), (140, 300, 1, 0, 200), (140, 2600, 1, 0, 2597), (140, 1200, 1, 500, 566),
]


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("nq,n,group,window,j", SPANS)
def test_any_bits_of_a_key_leave_the_queries_that_do_not_see_it(fmt, nq, n, group, window, j):
    # what page_write never stores, group scales past 64 and codes of -8, in a row whose scale is anything
    g = torch.Generator().manual_seed(nq + n)
    kv, table = m4.cache(g, [n], 1, fmt, 32)
    Q = torch.randn((nq, group, 128), generator=g).to(BF)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    page, row = int(table[0, j // 32]), j % 32
    was = [getattr(kv, name)[page, 0, row].clone() for name in m4.POOLS]
    spans = m4.seen(n, nq, window)
    blind = [i for i, (a, z) in enumerate(spans) if not a <= j < z]
    assert 0 < len(blind) < nq
    K, V = m4.pool_rows(kv, "k", table[0], n)[0], m4.pool_rows(kv, "v", table[0], n)[0]
    wide = [m4.attend_rows(Q[:, h].double(), K, V, blind, spans, F32, 0.0) for h in range(group)]
    narrow = [m4.attend_rows(Q[:, h].double(), K, V, blind, spans, BF, 2.0 ** -10 if nq * group > 16 else 0.0) for h in range(group)]
    # as large a scale as the reference lets stay below it
    near = 2.0 ** math.floor(math.log2(float(kv.v_scale[page, 0].nan_to_num().max()))) * JUST_BELOW_8
    rows = [(0x7E, 0x77, near), (0xFE, 0x99 if fmt is INT4 else 0xFF, near), (0x70, 0x77, 1.0), (0x68, 0x88, near),
            (0xE8, 0x88, near), (0x7E, 0x80, 0.0)]
    for trial in range(len(rows) + 24):
        if trial < len(rows):
            t, c, s = rows[trial]
            for name in m4.POOLS:
                x = getattr(kv, name)
                if name.endswith("scale"):
                    x[page, 0, row] = s
                else:
                    x.view(torch.uint8)[page, 0, row] = t if name.endswith("group") else c
        else:
            for name in m4.POOLS:
                x = getattr(kv, name)[page, 0, row]
                x = x.view(1) if x.dim() == 0 else x
                bits = x.view(torch.uint8)
                bits.copy_(torch.randint(0, 256, bits.shape, generator=g, dtype=torch.uint8))
        out, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32, return_lse=True)
        alone = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window)
        for h in range(group):
            tp._within(out[blind, h], wide[h][0], wide[h][2], "trial %d" % trial)
            tp._within(lse[blind, h], wide[h][1], wide[h][3], "lse, trial %d" % trial)
            tp._within(alone[blind, h], narrow[h][0], narrow[h][2], "alone, trial %d" % trial)
    for name, x in zip(m4.POOLS, was):
        getattr(kv, name)[page, 0, row] = x
    out = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8, E2M1, INT4])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("size", [2.0 ** 125, -3.4028234663852886e38])
def test_the_largest_scale_of_a_hidden_key_in_a_part_that_shows_a_query_nothing(fmt, size, which):
    # the keys are split: queries 30 and on of the first tile see keys of other parts than key 1487's only
    nq, n, group, window, page = 300, 1800, 2, 30, 128
    four = fmt in (E2M1, INT4)
    g = torch.Generator().manual_seed(7)
    kv, table = (m4.cache if four else tp._cache)(g, [n], 1, fmt, page)
    if four:
        K, V = (m4.pool_rows(kv, x, table[0], n)[0] for x in ("k", "v"))
    else:
        K, V = (pm.pool_rows(getattr(kv, x), getattr(kv, x + "_scale"), table[0], n, page)[0] for x in ("k", "v"))
    Q = torch.randn((nq, group, 128), generator=g).to(HF)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    top = {torch.float8_e4m3fn: 0x7E, torch.int8: 0x7F, E2M1: 0x77, INT4: 0x77}[fmt]
    at = (int(table[0, 1487 // page]), 0, 1487 % page)
    getattr(kv, which + "_scale")[at] = size
    getattr(kv, which).view(torch.uint8)[at] = top
    if four:
        getattr(kv, which + "_group").view(torch.uint8)[at] = 0x68   # 64
    spans = m4.seen(n, nq, window)
    blind = [i for i, (a, z) in enumerate(spans) if not a <= 1487 < z][::7]
    u_kv = 2.0 ** -10 if four else 2.0 ** -11
    for kw, u in ((dict(out_dtype=BF), u_kv), (dict(out_dtype=F32), 0.0), (dict(out_dtype=HF), 0.0)):
        for max_kv in (None, n):
            out = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, max_kv=max_kv, **kw)
            for h in range(group):
                want, _, bound, _ = m4.attend_rows(Q[:, h].double(), K, V, blind, spans, kw["out_dtype"], u)
                tp._within(out[blind, h], want, bound, "head %d" % h)
