"""GPU checks of attention over pages where a query sees nothing, or where what it does not see is
far from what it sees, against 64 bits."""
import math

import pytest
import torch

from tests import pages_model as pm
from tests import test_pages_gpu as tp
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu
BF, HF, F32, E4, I8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("fmt", [BF, HF, E4])
@pytest.mark.parametrize("nq,n,heads,causal", [(4680, 0, 12, False), (513, 100, 40, True), (700, 0, 3, True)])
def test_queries_that_see_no_key(fmt, nq, n, heads, causal):
    # a chunk before anything is cached, and more causal queries than cached tokens: whole tiles
    # of rows that see nothing are zeros, log-sum-exp -infinity, in every call
    g = _gen(nq)
    dtype = BF if fmt is E4 else fmt
    kv, table = tp._cache(g, [n], heads, fmt, 64)
    lens, table = torch.tensor([n], dtype=torch.int32).cuda(), table.cuda()
    Q = torch.randn((nq, heads, 128), generator=g).to(dtype).cuda()
    blind = nq - n if causal else nq
    first = None
    for _ in range(40):
        out, lse = api.page_attention(Q, kv, table, lens, causal=causal, return_lse=True)
        assert not out[:blind].any() and bool((lse[:blind] == -math.inf).all())
        assert bool(lse[blind:].isfinite().all())
        first = out if first is None else first
        assert torch.equal(out, first)


@pytest.mark.parametrize("nq,n,window", [(600, 600, 0), (777, 2000, 300)])
def test_masked_rows_keep_their_weight_sums(nq, n, window):
    # whole items of 16-bit pages under a mask: the rows' sums and the search for rows to do again
    # are exchanged by pairs of warps that run apart; every call gives the same, and values of one
    # give outputs of one, whatever the weights: a sum of n weights of at most 1 in fp32 and their
    # bf16 roundings (2^-8), then the output's (2^-8)
    g = _gen(nq + window)
    heads = 8
    kv, table = tp._cache(g, [n], heads, BF, 64)
    lens, table = torch.tensor([n], dtype=torch.int32).cuda(), table.cuda()
    Q = torch.randn((nq, heads, 128), generator=g).to(BF).cuda()
    want = api.page_attention(Q, kv, table, lens, window=window)
    for _ in range(100):
        assert torch.equal(api.page_attention(Q, kv, table, lens, window=window), want)
    kv.v.copy_(torch.where(kv.v.isnan(), kv.v, torch.ones_like(kv.v)))
    for _ in range(100):
        out = api.page_attention(Q, kv, table, lens, window=window)
        assert float((out.float() - 1).abs().max()) <= 2.0 ** -7 + n * 2.0 ** -23


def _seen(n, nq, window):
    """Keys [a, z) that each causal query sees."""
    pos = [n - nq + i for i in range(nq)]
    return [(max(0, p + 1 - window) if window else 0, max(0, p + 1)) for p in pos]


def _check_lse(Q, kv, table, n, window, lse):
    """Every row's log-sum-exp against 64 bits over the keys that it sees and no others."""
    K = pm.pool_rows(kv.k, kv.k_scale, table[0].cpu(), n, kv.page_tokens)[0]
    for i, (a, z) in enumerate(_seen(n, Q.shape[0], window)):
        for hq in range(Q.shape[1]):
            _, want, _, bound = pm.attend(Q[i:i + 1, hq].double().cpu(), K[a:z], K[a:z], 128 ** -0.5, False, 0, 2.0 ** -11, F32)
            tp._within(lse[i:i + 1, hq], want, bound, "lse %d head %d" % (i, hq))


SPANS = [  # queries, cached tokens, query heads, window, a key that only some queries see
    (5, 300, 2, 0, 297), (16, 2000, 1, 0, 1990), (7, 900, 2, 300, 596), (140, 300, 1, 0, 297),
    (140, 300, 1, 0, 200), (140, 2600, 1, 0, 2597), (140, 1200, 1, 500, 566), (300, 300, 1, 0, 131),
]


@pytest.mark.parametrize("fmt", [E4, I8])
@pytest.mark.parametrize("nq,n,group,window,j", SPANS)
def test_a_value_that_is_not_finite_leaves_the_log_sum_exp(fmt, nq, n, group, window, j):
    # the log-sum-exp is of the scores alone, whole or split, few rows or many
    g = _gen(nq + n)
    kv, table = tp._cache(g, [n], 1, fmt, 32)
    Q = torch.randn((nq, group, 128), generator=g).to(BF)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    kv.v_scale[int(table[0, j // 32]), 0, j % 32] = math.nan
    out, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32, return_lse=True)
    for i, (a, z) in enumerate(_seen(n, nq, window)):
        assert bool(out[i].isnan().all()) if a <= j < z else bool(out[i].isfinite().all())
    _check_lse(Q, kv, table, n, window, lse)


def _check_rows(Q, kv, table, n, window, rows, out, lse=None, u_kv=0.0):
    """Rows against 64 bits over the keys that each sees and no others, so that a bound knows no
    other keys' sizes either."""
    group = Q.shape[1] // kv.heads
    u_p = pm.HALF_EPS[HF if kv.k.dtype in pm.TOP else Q.dtype]
    seen = _seen(n, Q.shape[0], window)
    for h in range(kv.heads):
        K = pm.pool_rows(kv.k, kv.k_scale, table[0].cpu(), n, kv.page_tokens)[h]
        V = pm.pool_rows(kv.v, kv.v_scale, table[0].cpu(), n, kv.page_tokens)[h]
        for i in rows:
            a, z = seen[i]
            for hq in range(h * group, (h + 1) * group):
                want, want_lse, bound, lse_bound = pm.attend(Q[i:i + 1, hq].double().cpu(), K[a:z], V[a:z], 128 ** -0.5,
                                                             False, 0, u_p, out.dtype, u_kv, u_kv)
                tp._within(out[i:i + 1, hq], want, bound, "row %d head %d" % (i, hq))
                if lse is not None:
                    tp._within(lse[i:i + 1, hq], want_lse, lse_bound, "lse %d head %d" % (i, hq))


@pytest.mark.parametrize("fmt", [E4, I8])
@pytest.mark.parametrize("nq,n,group,window,j", SPANS)
@pytest.mark.parametrize("which,size", [("v", math.inf), ("v", 2.0 ** 40), ("v", 2.0 ** 20), ("v", math.nan),
                                        ("k", 2.0 ** 40), ("k", math.nan)])
def test_scales_of_keys_that_some_queries_do_not_see(fmt, nq, n, group, window, j, which, size):
    # a key far larger than all that the other queries see
    g = _gen(nq + n)
    kv, table = tp._cache(g, [n], 1, fmt, 32)
    Q = torch.randn((nq, group, 128), generator=g).to(BF)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    getattr(kv, which + "_scale")[int(table[0, j // 32]), 0, j % 32] = size
    out, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32, return_lse=True)
    alone = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window)
    sees = [i for i, (a, z) in enumerate(_seen(n, nq, window)) if a <= j < z]
    blind = [i for i in range(nq) if i not in sees]
    assert blind and sees
    rows = range(nq) if math.isfinite(size) and which == "v" else blind
    _check_rows(Q, kv, table, n, window, rows, out, lse)
    _check_rows(Q, kv, table, n, window, rows, alone, u_kv=0.0 if nq * group <= 16 else 2.0 ** -11)
    if not math.isfinite(size):
        assert not bool(out[sees].isfinite().any()) and not bool(alone[sees].isfinite().any())
        if which == "k":
            assert bool(lse[sees].isnan().all())


@pytest.mark.parametrize("fmt", [BF, HF, E4, I8])
@pytest.mark.parametrize("nq,n", [(3, 300), (140, 300), (140, 2600)])
def test_scores_far_past_the_exponential(fmt, nq, n):
    # scores of 2^30 and more, where fp32 steps are whole powers of two: a query's largest score
    # has all the weight, and the output is its value, to the roundings of weight, value and output
    g = _gen(nq + n)
    kv, table = tp._cache(g, [n], 1, fmt, 32)
    dtype = HF if fmt is HF else BF
    Q = torch.randn((nq, 2, 128), generator=g).to(dtype)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    scale = 3.0e8
    K = pm.pool_rows(kv.k, kv.k_scale, table[0], n, 32)[0]
    V = pm.pool_rows(kv.v, kv.v_scale, table[0], n, 32)[0]
    s = torch.einsum("ihd,jd->hij", Q.double(), K) * scale
    seen = torch.arange(n)[None] <= torch.arange(n - nq, n)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    two = s.topk(2, -1).values
    # the gap to the second is thousands of the score's roundings for all but a few rows
    clear = two[..., 0] - two[..., 1] > 128 * 2.0 ** -22 * (Q.double().abs().amax() * K.abs().amax() * 128 * scale)
    assert float(clear.double().mean()) > 0.5
    want = V[s.argmax(-1)]
    for kw in (dict(), dict(return_lse=True, out_dtype=F32)):
        out = api.page_attention(Q.cuda(), kv, table.cuda(), lens, scale=scale, **kw)
        if kw:
            out, lse = out
            assert float(((lse.cpu().double().T - two[..., 0]) / two[..., 0].abs()).abs().max()) <= 2.0 ** -16
        assert bool(out.isfinite().all())
        off = (out.double().cpu().transpose(0, 1) - want).abs()
        assert float(off[clear].max()) <= 3 * 2.0 ** -8 * float(V.abs().max())


def _time(f):
    f()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("nq,n,heads,window", [(1, 20000, 4, 0), (4, 20000, 4, 0), (300, 6000, 2, 0), (300, 6000, 2, 1000),
                                               (64, 9000, 1, 0)])
def test_a_visible_value_that_is_not_finite_costs_little(nq, n, heads, window):
    # only rows that such a value spoilt without being seen are done again; done again key by key,
    # all rows that see it would take more than thirty times as long
    g = _gen(nq)
    kv, table = tp._cache(g, [n], heads, BF, 64)
    lens, table = torch.tensor([n], dtype=torch.int32).cuda(), table.cuda()
    Q = torch.randn((nq, heads, 128), generator=g).to(BF).cuda()

    def call():
        return api.page_attention(Q, kv, table, lens, window=window, return_lse=True)
    clean, clean_lse = call()
    clean_time = min(_time(call) for _ in range(3))
    j = n - nq - (window // 2) if window else 70  # seen by every query
    kv.v[int(table[0, j // 64]), :, j % 64, 9] = math.inf
    kv.v[int(table[0, j // 64]), :, j % 64, 10] = math.nan
    out, lse = call()
    keep = [c for c in range(128) if c not in (9, 10)]
    assert torch.equal(out[..., keep], clean[..., keep]) and torch.equal(lse, clean_lse)
    assert bool((out[..., 9] == math.inf).all()) and bool(out[..., 10].isnan().all())
    assert min(_time(call) for _ in range(3)) <= 8 * clean_time


@pytest.mark.parametrize("nq,n,group,window,j", SPANS + [(5, 15000, 8, 0, 14998)])
def test_nan_codes_of_keys_that_some_queries_do_not_see(nq, n, group, window, j):
    # E4M3 has codes that are NaN; page_write stores none, but pages may come from elsewhere
    g = _gen(nq + n)
    kv, table = tp._cache(g, [n], 1, E4, 32)
    Q = torch.randn((nq, group, 128), generator=g).to(BF)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    kv.v.view(torch.uint8)[int(table[0, j // 32]), 0, j % 32, 5] = 0x7F
    kv.v.view(torch.uint8)[int(table[0, j // 32]), 0, j % 32, 77] = 0xFF
    out, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32, return_lse=True)
    alone = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window)
    sees = [i for i, (a, z) in enumerate(_seen(n, nq, window)) if a <= j < z]
    blind = [i for i in range(nq) if i not in sees]
    assert blind and sees
    _check_rows(Q, kv, table, n, window, blind, out, lse)
    _check_rows(Q, kv, table, n, window, blind, alone, u_kv=0.0 if nq * group <= 16 else 2.0 ** -11)
    keep = [c for c in range(128) if c not in (5, 77)]
    for o in (out, alone):
        assert bool(o[sees][..., [5, 77]].isnan().all()) and bool(o[sees][..., keep].isfinite().all())
    _check_lse(Q, kv, table, n, window, lse)
    kv.k.view(torch.uint8)[int(table[0, j // 32]), 0, j % 32, 5] = 0x7F
    out = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32)
    assert bool(out[sees].isnan().all())
    _check_rows(Q, kv, table, n, window, blind, out)


UNLIKE = [  # q lengths, cached lengths, q heads, heads, type, format, page, causal, window
    ([5, 0, 200, 1, 0, 60], [900, 700, 3000, 1, 0, 2000], 4, 2, BF, BF, 32, True, 0),
    ([0, 0, 290], [10, 0, 2000], 1, 1, HF, HF, 64, False, 0),
    ([1 + b % 3 if b % 5 else 0 for b in range(69)] + [130], [3 * b + 3 for b in range(69)] + [1700], 20, 1, BF, I8, 16, True, 0),
    ([100, 0, 0, 70], [1500, 0, 0, 2100], 3, 3, BF, E4, 128, True, 600),
]


@pytest.mark.parametrize("case", UNLIKE)
def test_split_items_of_unlike_sequences(case):
    q_lens, kv_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    g = _gen(sum(q_lens))
    kv, table = tp._cache(g, kv_lens, heads, fmt, page)
    Q = torch.randn((sum(q_lens), q_heads, 128), generator=g).to(dtype)
    tp._check(Q, kv, table, kv_lens, q_lens, causal, window)
    # any of them may be the longest, as far as the call knows
    tp._check(Q, kv, table, kv_lens, q_lens, causal, window, max_q=sum(q_lens))


def test_split_items_report_bad_arguments():
    g = _gen(4)
    kv, table = tp._cache(g, [2000, 5, 900], 1, BF, 32)
    Q = torch.randn((130, 1, 128), generator=g).to(BF).cuda()

    def status_of(cu=(0, 90, 90, 130), lens=(2000, 5, 900), max_q=130):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(Q, 7.0)
        api.page_attention(Q, kv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), max_q=max_q,
                           cu_q=torch.tensor(cu, dtype=torch.int32).cuda(), status=st, out=out)
        return int(st), out
    st, good = status_of()
    assert st == 0 and not bool((good == 7).all(-1).any())
    for bad in (dict(cu=(0, 130, 0, 130)), dict(cu=(0, 90, 90, 140)), dict(cu=(-2, 90, 90, 130)), dict(lens=(2000, -5, 900)),
                dict(lens=(2000, 5, 99999)), dict(max_q=80)):
        st, out = status_of(**bad)
        assert st == qvg.QVG_DEV_BAD_INDEX, bad
    st, out = status_of(lens=(2000, -5, 900))  # a sequence without queries, cut
    assert torch.equal(out, good)
    st, out = status_of(max_q=80)
    assert bool((out[80:90] == 7).all()) and torch.equal(out[90:], good[90:])


SHARED = [  # cached lengths, q lengths (in turn), q heads, heads, q type, format, page, causal, window
    ([2900, 0, 1, 64, 127, 128, 129, 700] * 3, [1], 8, 4, BF, E4, 64, True, 0),
    ([300, 900, 40, 2000], [1, 2], 48, 24, HF, I8, 16, True, 250),   # a window that begins in the middle
    ([2000, 1500] * 2, [5], 60, 30, BF, E4, 32, True, 700),
    ([17] * 11, [1], 8, 8, BF, I8, 16, True, 0),                     # fewer stages than shares would like
    ([0, 0, 0, 0], [1, 0], 40, 40, BF, E4, 16, False, 0),            # no keys: a stage each where there is a query
    ([0, 0, 0, 0], [0, 0, 1, 0], 40, 40, HF, I8, 16, False, 0),
    ([300, 20], [0], 100, 100, BF, I8, 16, True, 0),                 # no stages at all (one query follows)
    ([64] * 304, [1], 2, 1, HF, I8, 64, True, 0),                    # one stage a head, four a share
    ([65] * 152, [1], 4, 2, BF, E4, 32, True, 0),
]


@pytest.mark.parametrize("case", SHARED)
def test_equal_shares_of_8_bit_keys(case):
    # the keys of all heads cut into equal shares, and the sizes where shares and stages nearly
    # run out; the workspace says that the call takes this way
    kv_lens, q_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    q_lens = [q_lens[b % len(q_lens)] for b in range(len(kv_lens))]
    if not any(q_lens):
        kv_lens, q_lens = kv_lens + [5], q_lens + [1]
    g = _gen(sum(q_lens) + sum(kv_lens) + heads)
    kv, table = tp._cache(g, kv_lens, heads, fmt, page)
    cells = heads * len(kv_lens)
    assert 76 < cells <= 608
    longest = 1 + 152 * 2 * 2048 // cells
    wide = torch.zeros((len(kv_lens), max(table.shape[1], -(-longest // page))), dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    prm = qvg.qvg_page_attention_params(
        n_seqs=len(kv_lens), n_q_heads=q_heads, n_heads=heads, d=128, page_tokens=page, format=kv.format,
        q_dtype=api._DT[dtype], out_dtype=api._DT[dtype], n_pages=kv.n_pages, max_pages=wide.shape[1], causal=int(causal),
        window=window, total_q=sum(q_lens), max_q=max(q_lens), max_kv=longest, scale=0.1, q_token_stride=q_heads * 128,
        q_head_stride=128, o_token_stride=q_heads * 128, o_head_stride=128)
    assert qvg.qvg_page_attention_workspace_bytes(prm) == 2 * 304 * 16 * (128 + 2) * 4 + cells * 8
    Q = (1.5 * torch.randn((sum(q_lens), q_heads, 128), generator=g)).to(dtype)
    tp._check(Q, kv, wide, kv_lens, q_lens, causal, window, max_kv=longest)


@pytest.mark.parametrize("fmt", [E4, I8])
@pytest.mark.parametrize("window", [0, 400])
def test_hidden_keys_in_equal_shares(fmt, window):
    # five queries of 40 heads over shares that end anywhere: a scale, and a NaN code, of a key that
    # only the last two queries see
    g = _gen(window + 1)
    n, heads, nq = 1900, 40, 5
    kv, table = tp._cache(g, [n, n], heads, fmt, 32)
    longest = 1 + 152 * 2 * 2048 // (2 * heads)
    wide = torch.zeros((2, -(-longest // 32)), dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    Q = torch.randn((2 * nq, heads, 128), generator=g).to(BF)
    lens = torch.tensor([n, n], dtype=torch.int32).cuda()

    def call():
        return api.page_attention(Q.cuda(), kv, wide.cuda(), lens, max_kv=longest, window=window, out_dtype=F32, return_lse=True)
    clean, clean_lse = call()
    page, row = int(table[0, (n - 2) // 32]), (n - 2) % 32
    for size in (2.0 ** 40, math.inf, math.nan):
        was = kv.v_scale[page, :, row].clone()
        kv.v_scale[page, :, row] = size
        out, lse = call()
        assert torch.equal(out[:3], clean[:3]) and torch.equal(out[5:], clean[5:]) and torch.equal(lse, clean_lse)
        if not math.isfinite(size):
            assert not bool(out[3:5].isfinite().any())
        kv.v_scale[page, :, row] = was
    if fmt is E4:
        kv.v.view(torch.uint8)[page, :, row, 7] = 0x7F
        out, lse = call()
        # (rows done again: each is within its roundings, fp16 weights, of the same value)
        near = 8 * 2.0 ** -11 * float(pm.pool_rows(kv.v, kv.v_scale, table[0], n - 2, 32).abs().max())
        assert float((out[:3] - clean[:3]).abs().max()) <= near and torch.equal(out[5:], clean[5:])
        assert bool(out[3:5][..., 7].isnan().all()) and int(out.isnan().sum()) == 2 * heads
        assert float((lse - clean_lse).abs().max()) <= 2.0 ** -12


@pytest.mark.parametrize("nq,n,window", [(300, 6000, 0), (64, 9000, 0), (300, 6000, 3000)])
@pytest.mark.parametrize("lse", [False, True])
def test_a_large_scale_that_all_have_seen_before_costs_little(nq, n, window, lse):
    # a value sixty times the nearest ones among the newest keys, and as large a one that every
    # query sees far back: no query needs to be done again
    g = _gen(nq + n)
    kv, table = tp._cache(g, [n], 2, E4, 64)
    lens, table = torch.tensor([n], dtype=torch.int32).cuda(), table.cuda()
    Q = torch.randn((nq, 2, 128), generator=g).to(BF).cuda()

    def call():
        return api.page_attention(Q, kv, table, lens, window=window, return_lse=lse)
    call()
    clean_time = min(_time(call) for _ in range(3))
    for j in (n - window + 5 if window else 70, n - 3):
        kv.v_scale[int(table[0, j // 64]), :, j % 64] *= 60.0
    call()
    assert min(_time(call) for _ in range(3)) <= 8 * clean_time
