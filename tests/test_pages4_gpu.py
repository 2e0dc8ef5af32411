"""GPU checks of the 4-bit pages against their definition in 64 bits (pages4_model.py): rows written and
read back, and attention over them by both kernels, at the sizes, layouts and masks where they can go
wrong.

Memory that no sequence reaches holds any codes, and NaN in both kinds of scales.
"""
import math

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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- rows written and read

WRITE = [  # tokens, heads, dtype, format, page, turned channels (0: none), interleaved
    (1, 1, BF, E2M1, 16, 128, False),
    (5, 3, HF, INT4, 16, 0, False),
    (67, 7, F32, E2M1, 32, 0, False),
    (67, 12, BF, INT4, 64, 128, True),
    (131, 4, F32, INT4, 128, 64, False),
    (40, 5, HF, E2M1, 64, 0, False),
    (129, 9, BF, E2M1, 128, 96, False),
    (33, 2, F32, INT4, 32, 0, False),
    (20, 6, HF, E2M1, 16, 32, True),
    (300, 8, BF, INT4, 64, 0, False),
    (19, 5, BF, E2M1, 16, 24, False),   # turned halves that begin inside a group
    (21, 4, F32, INT4, 16, 120, False),
    (21, 4, HF, E2M1, 32, 8, True),
]


def _blank(pages, heads, page, fmt):
    kv = api.allocate_pages(pages, heads, page, fmt)
    for t in (kv.k, kv.v, kv.k_group, kv.v_group):
        t.view(torch.uint8).fill_(0x11)
    kv.k_scale.fill_(-1.0)
    kv.v_scale.fill_(-1.0)
    return kv


@pytest.mark.parametrize("case", WRITE)
def test_write_and_read(case):
    n, heads, dtype, fmt, page, rot, inter = case
    g = _gen(n + heads)
    rows = torch.randn((n, 2 * heads, 128), generator=g)
    rows[..., 3::50] += 30.0
    rows[0, 0, 32:48] = 0.0                       # a group of zeros
    rows[-1, -1] *= 2.0 ** -12 * torch.arange(128) / 128   # magnitudes rising through the row
    rows[-1, -1, -1] = 1.0                        # groups far below the largest: small or zero scales
    rows = rows.to(dtype)
    K, V = rows[:, :heads], rows[:, heads:]
    kv = _blank(-(-n // page) + 3, heads, page, fmt)
    order = torch.randperm(kv.n_pages, generator=g)
    i = torch.arange(n)
    slots = order[i // page] * page + i % page
    table = pos = None
    want_k, err_k = K.double(), torch.zeros(K.shape, dtype=torch.float64)
    if rot:
        freqs, _ = api.rope_frequencies(rot)
        table = api.rope_table(rot, freqs=freqs, interleaved=inter)
        pos = torch.randint(0, 50000, (1, n), generator=_gen(1))
        want_k, err_k = pm.rotate(K, pos, freqs.tolist(), table.sections, inter)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = rows.cuda()
    api.page_write(kv, rows[:, :heads], rows[:, heads:], slots.cuda(), rope=table,
                   positions=None if pos is None else pos.cuda(), status=status)
    top = m4.TOP[fmt]

    def flat(t):  # [slot][heads][..]
        return t.view(torch.uint8 if t.element_size() == 1 else t.dtype).transpose(1, 2).flatten(0, 1).cpu()
    for name, x64, err in (("k", want_k, err_k), ("v", V.double(), torch.zeros_like(err_k))):
        raw, s = flat(getattr(kv, name)), flat(getattr(kv, name + "_scale"))
        t = flat(getattr(kv, name + "_group"))
        rest = torch.ones(len(s), dtype=torch.bool)
        rest[slots] = False
        assert bool((raw[rest] == 0x11).all()) and bool((t[rest] == 0x11).all()) and bool((s[rest] == -1).all())
        raw, s, t = raw[slots], s[slots], t[slots].view(torch.float8_e4m3fn)
        exact = not (rot and name == "k")
        if exact and dtype is not F32:  # every quotient correctly rounded: the definition's bits
            want = m4.stored(x64, fmt)
            assert torch.equal(raw & 0x77 if fmt is E2M1 else raw, want[0] & 0x77 if fmt is E2M1 else want[0])
            assert torch.equal(t.float(), want[1].float())
            assert torch.equal(m4.decoded(raw, t, s, fmt), m4.decoded(*want, fmt))
        e = err.amax(-1)
        a = x64.abs().amax(-1)
        # the scale is one rounding of a / (64 top), a known to e
        tp._within(s, a / (64 * top), (a * 2.0 ** -24 + e) * (1 + 2.0 ** -20) / (64 * top), "scale")
        # group scales: half an E4M3 step (2^-4 of it, or of 2^-9) of 64 a_g / a, which is known to
        # err / a and three roundings
        ag = x64.abs().unflatten(-1, (8, 16)).amax(-1)
        q = 64 * ag / a[..., None]
        slack = 64 * 2 * e[..., None] / a[..., None] + q * 2.0 ** -22
        tp._within(t.float(), q, torch.maximum(q * 2.0 ** -4, torch.tensor(2.0 ** -10)) + slack, "group scale")
        # each value is as near to x as any code of its scales, but for what fp32 loses: the turned
        # channel's error and four roundings of a quotient of at most 11
        unit = (t.double() * s.double()[..., None]).repeat_interleave(16, -1)
        y = m4.decoded(raw, t, s, fmt)
        best = torch.full(y.shape, math.inf, dtype=torch.float64)
        for v in m4.VALUES[fmt][:8] + m4.VALUES[fmt][-7:]:
            best = torch.minimum(best, (v * unit - x64).abs())
        assert bool(((y - x64).abs() <= best + 2 * err + 2 * e[..., None] + unit * 11 * 2.0 ** -21).all())
    # read back: whole, and a part that begins and ends inside pages
    tab = torch.full((2, kv.n_pages), -7, dtype=torch.int32)
    tab[0, :-(-n // page)] = order[:-(-n // page)].to(torch.int32)
    lens = torch.tensor([n, 0], dtype=torch.int32).cuda()
    for out_dtype in (BF, HF, F32):
        for first, count in ((0, n), (n // 3, n), (n, 5)):
            X = api.page_read(kv, tab.cuda(), lens, count, first=first, out_dtype=out_dtype, status=status)
            assert X.shape == (2, 2 * heads, count, 128)
            for which, name in enumerate(("k", "v")):
                want = m4.pool_rows(kv, name, tab[0], n)[:, first:first + count]
                have = want.shape[1]
                bound = want.abs() * (pm.HALF_EPS[out_dtype] + 2.0 ** -24) + pm.TINY[out_dtype]
                tp._within(X[0, which::2, :have], want, bound, "read")
                assert not X[0, which::2, have:].any() and not X[1].any()
    assert int(status) == 0


@pytest.mark.parametrize("fmt", [E2M1, INT4])
def test_write_skips_and_reports(fmt):
    heads, page = 3, 16
    kv = _blank(4, heads, page, fmt)
    K = torch.randn((6, heads, 128), generator=_gen(2)).cuda()
    V = torch.randn((6, heads, 128), generator=_gen(3)).cuda()
    K[1, 0, 7] = float("nan")
    V[2, 2, 0] = float("-inf")
    K[3, 1] = 0.0
    V[3, 1] = 2.0 ** -101
    K[5] *= 2.0 ** 120           # near the largest and the smallest rows that are stored
    V[5] *= 2.0 ** -97
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.page_write(kv, K, V, torch.tensor([-1, 17, 18, 19, 4 * page, 20]).cuda(), status=status)
    assert int(status) == qvg.QVG_DEV_NONFINITE | qvg.QVG_DEV_BAD_INDEX
    ks, vs = kv.k_scale.cpu(), kv.v_scale.cpu()
    assert int((ks == -1).sum()) == int((vs == -1).sum()) == (4 * page - 4) * heads
    assert int(ks.isnan().sum()) == int(vs.isnan().sum()) == 1
    assert bool(ks[1, 0, 1].isnan()) and bool(vs[1, 2, 2].isnan())
    for pool in (kv.v, kv.v_group):
        assert not pool[1, 1, 3].view(torch.uint8).any() and not pool[1, 2, 2].view(torch.uint8).any()
    assert ks[1, 1, 3] == 0 and vs[1, 1, 3] == 0
    tab = torch.tensor([[1]], dtype=torch.int32).cuda()
    X = api.page_read(kv, tab, torch.tensor([5], dtype=torch.int32).cuda(), 5, out_dtype=F32)
    assert bool(X[0, 0, 1].isnan().all()) and bool(X[0, 5, 2].isnan().all())
    assert int(X[:, :, 1:4].isnan().sum()) == 2 * 128
    for which, x in ((0, K[5]), (1, V[5])):
        want = m4.decoded(*m4.stored(x.cpu(), fmt), fmt)
        # one code apart at most where a quotient, four roundings off, lies at a border
        unit = x.abs().amax(-1, keepdim=True).double().cpu() / m4.TOP[fmt]
        off = (X[0, which::2, 4].double().cpu() - want).abs()
        assert bool((off <= 2.01 * unit).all()) and float((off > unit * 2.0 ** -20).double().mean()) < 0.01
    status.zero_()
    api.page_write(kv, K[:0], V[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), status=status)
    assert int(status) == 0


def test_read_of_bad_tables_and_lengths():
    kv = _blank(3, 2, 16, INT4)
    K = torch.ones((48, 2, 128), device="cuda")
    api.page_write(kv, K, 2 * K, torch.arange(48).cuda())
    tab = torch.tensor([[2, 9], [-3, 1]], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    X = api.page_read(kv, tab, torch.tensor([20, 99], dtype=torch.int32).cuda(), 40, status=status)
    assert int(status) == qvg.QVG_DEV_BAD_INDEX
    assert bool((X[0, 0, :16] == 1).all()) and not X[0, :, 16:].any()
    assert not X[1, :, :16].any() and bool((X[1, 1, 16:32] == 2).all()) and not X[1, :, 32:].any()


def test_strided_and_broadcast_rows():
    g = _gen(21)
    n, heads, page = 50, 4, 16
    i = torch.arange(n).cuda()
    wide = torch.randn((n, 3 * heads, 128), generator=g).to(BF).cuda()
    one = torch.randn((n, 1, 128), generator=g).to(BF).cuda().expand(n, heads, 128)
    a, b = _blank(4, heads, page, E2M1), _blank(4, heads, page, E2M1)
    api.page_write(a, wide[:, heads:2 * heads], one, i)
    api.page_write(b, wide[:, heads:2 * heads].contiguous(), one.contiguous(), i)
    for x, y in zip((a.k, a.v, a.k_group, a.v_group), (b.k, b.v, b.k_group, b.v_group)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


# ---------------------------------------------------------------- attention

def _check(Q, kv, table, kv_lens, q_lens, causal, window, scale=None, out_dtype=None, **kw):
    group = Q.shape[1] // kv.heads
    cu = torch.tensor([sum(q_lens[:b]) for b in range(len(q_lens) + 1)], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(dict(cu_q=cu.cuda(), max_q=max(q_lens), max_kv=max(kv_lens)), **kw)
    lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
    got, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, causal=causal, window=window, scale=scale,
                                  out_dtype=out_dtype, return_lse=True, status=status, **kw)
    alone = api.page_attention(Q.cuda(), kv, table.cuda(), lens, causal=causal, window=window, scale=scale,
                               out_dtype=out_dtype, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    # without the log-sum-exp and with a bf16 output, keys and values may meet many rows rounded to fp16, once
    # as a group's scale times a row's and once more as that times the code
    u_kv = 2.0 ** -10 if got.dtype is BF and max(q_lens) * group > 16 else 0.0
    if not u_kv:
        assert torch.equal(alone, got)
    Qc = Q.double().cpu()
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        if nq == 0:
            continue
        K, V = m4.pool_rows(kv, "k", table[b], n), m4.pool_rows(kv, "v", table[b], n)
        rows = slice(int(cu[b]), int(cu[b]) + nq)
        for hq in range(Q.shape[1]):
            args = (Qc[rows, hq], K[hq // group], V[hq // group], 128 ** -0.5 if scale is None else scale, causal, window,
                    2.0 ** -11, got.dtype)
            want, want_lse, bound, lse_bound = pm.attend(*args)
            tp._within(got[rows, hq], want, bound, "sequence %d head %d" % (b, hq))
            if u_kv:
                tp._within(alone[rows, hq], want, pm.attend(*args, u_kv, u_kv)[2], "alone: sequence %d head %d" % (b, hq))
            none = want_lse == -math.inf
            assert torch.equal(lse[rows, hq].cpu() == -math.inf, none)
            tp._within(lse[rows, hq].cpu()[~none], want_lse[~none], lse_bound[~none], "lse")
    return got, lse


ATTEND = [  # q lengths, cached lengths, q heads, heads, q type, format, page, causal, window
    ([1], [1], 1, 1, BF, E2M1, 16, True, 0),
    ([1, 1, 1], [5, 0, 300], 8, 2, BF, INT4, 16, True, 0),      # an empty sequence sees nothing
    ([1] * 4, [33, 64, 1000, 127], 4, 4, HF, E2M1, 32, True, 0),
    ([1, 1], [4000, 517], 16, 2, BF, INT4, 64, True, 0),          # splits
    ([1, 1], [3900, 40], 7, 1, HF, INT4, 128, True, 700),
    ([3, 5, 2], [3, 200, 77], 4, 2, HF, E2M1, 16, True, 0),
    ([4, 2], [2, 90], 3, 3, BF, INT4, 16, True, 0),               # first rows see nothing
    ([2, 0, 7], [900, 10, 450], 6, 2, BF, E2M1, 32, False, 0),    # sixteen rows at most: two groups of eight
    ([5], [1000], 6, 2, HF, INT4, 16, True, 300),
    ([70], [70], 2, 2, BF, E2M1, 64, True, 0),
    ([129, 17], [513, 17], 4, 1, HF, INT4, 16, True, 100),
    ([200], [391], 2, 2, BF, INT4, 128, False, 0),
    ([300, 1, 45], [300, 700, 1000], 8, 4, BF, E2M1, 32, True, 0),
    ([260], [1300], 3, 1, HF, INT4, 64, False, 0),
    ([150], [1200], 2, 1, HF, E2M1, 64, True, 64),
    ([257], [257], 1, 1, BF, INT4, 16, False, 33),                # a window without causality
    ([64], [3000], 1, 1, BF, E2M1, 64, True, 0),                  # many splits of one tile
    ([31], [31], 128, 1, BF, INT4, 16, True, 0),                  # 128 query heads share one
    ([513], [640], 5, 5, HF, E2M1, 128, True, 0),
    ([257], [1100], 77, 77, BF, INT4, 64, True, 0),               # more than a round: whole items, split ones
    ([40, 20], [2500, 900], 2, 2, HF, E2M1, 16, True, 0),         # few items of unlike sequences: all split
    ([2], [5000], 8, 1, BF, E2M1, 128, True, 3000),               # 16 rows, splits through memory
    ([300, 0, 70, 513], [400, 50, 70, 1200], 44, 44, BF, E2M1, 32, True, 0),   # those that see the most first
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention(case):
    q_lens, kv_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    g = _gen(sum(q_lens) + sum(kv_lens))
    kv, table = m4.cache(g, kv_lens, heads, fmt, page)
    Q = (1.5 * torch.randn((sum(q_lens), q_heads, 128), generator=g)).to(dtype)
    _check(Q, kv, table, kv_lens, q_lens, causal, window)


SHARES = [  # cached lengths, q lengths (in turn), q heads, heads, q type, format, page, causal, window
    ([2900, 0, 1, 64, 127, 128, 129, 700] * 3, [1], 8, 4, BF, E2M1, 64, True, 0),
    ([300, 900, 40, 2000], [1, 2], 48, 24, HF, INT4, 16, True, 250),   # a window that begins in the middle
    ([2000, 1500] * 2, [5], 60, 30, BF, E2M1, 32, True, 700),
    ([17] * 11, [1], 8, 8, BF, INT4, 16, True, 0),                     # fewer stages than shares would like
    ([0, 0, 0, 0], [1, 0], 40, 40, BF, E2M1, 16, False, 0),            # no keys: a stage each where there is a query
    ([128] * 304, [1], 2, 1, HF, INT4, 64, True, 0),                   # one stage a head
    ([129] * 152, [1], 4, 2, BF, E2M1, 32, True, 0),
    ([5, 3, 2500], [4], 90, 30, HF, INT4, 128, True, 0),               # 12 rows; some see nothing
]


@pytest.mark.parametrize("case", SHARES)
def test_attention_in_equal_shares(case):
    kv_lens, q_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    q_lens = [q_lens[b % len(q_lens)] for b in range(len(kv_lens))]
    g = _gen(sum(q_lens) + sum(kv_lens) + heads)
    kv, table = m4.cache(g, kv_lens, heads, fmt, page)
    longest = 1 + 152 * 2 * 2048 // (heads * len(kv_lens))
    wide = torch.zeros((len(kv_lens), max(table.shape[1], -(-longest // page))), dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    Q = (1.5 * torch.randn((sum(q_lens), q_heads, 128), generator=g)).to(dtype)
    _check(Q, kv, wide, kv_lens, q_lens, causal, window, max_kv=longest)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("nq,fmt", [(1, E2M1), (40, INT4)])
def test_attention_lengths(n, nq, fmt):
    nq = min(n, nq)
    g = _gen(1000 + n)
    kv, table = m4.cache(g, [n], 1, fmt, 16)
    Q = torch.randn((nq, 3, 128), generator=g).to(BF)
    _check(Q, kv, table, [n], [nq], True, 0)
    _check(Q, kv, table, [n], [nq], False, 0)


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("nq", [2, 60])
def test_strides_types_and_default_arguments(fmt, nq):
    g = _gen(8)
    kv_lens, q_lens = [150, 300], [nq, nq]
    kv, table = m4.cache(g, kv_lens, 2, fmt, 32)
    wide = torch.randn((2 * nq, 12, 128), generator=g).to(HF).cuda()
    Q = wide[:, 2:6]
    plain, _ = _check(Q, kv, table, kv_lens, q_lens, True, 0)
    for out_dtype in (BF, F32, HF):
        _check(Q, kv, table, kv_lens, q_lens, True, 0, out_dtype=out_dtype)
    lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
    out = torch.zeros((4, 2 * nq, 128), dtype=HF, device="cuda").transpose(0, 1)
    assert api.page_attention(Q, kv, table.cuda(), lens, out=out, max_kv=300) is out and torch.equal(out, plain)
    _check(Q, kv, table, kv_lens, q_lens, True, 0, max_kv=None, max_q=None)
    _check(Q, kv, table, kv_lens, q_lens, True, 0, scale=-0.3)
    _check(Q, kv, table, kv_lens, q_lens, True, 0, scale=0.0)
    one = torch.randn((2 * nq, 1, 128), generator=g).to(HF).cuda().expand(2 * nq, 4, 128)
    _check(one, kv, table, kv_lens, q_lens, True, 0)


@pytest.mark.parametrize("nq", [1, 60])
@pytest.mark.parametrize("fmt", [E2M1, INT4])
def test_value_scales_of_many_sizes(nq, fmt):
    g = _gen(14)
    n, page = 700, 16
    for order in ("rising", "falling", "mixed"):
        kv, table = m4.cache(g, [n], 1, fmt, page)
        e = torch.linspace(-60, 60, n) * (-1 if order == "falling" else 1)
        if order == "mixed":
            e = e[torch.randperm(n, generator=g)]
        for j in range(n):
            kv.v_scale[int(table[0, j // page]), 0, j % page] = 2.0 ** float(e[j])
        Q = torch.randn((nq, 2, 128), generator=g).to(HF)
        _check(Q, kv, table, [n], [nq], True, 0, out_dtype=F32)


@pytest.mark.parametrize("nq,fmt", [(1, E2M1), (90, E2M1), (90, INT4)])
def test_groups_of_many_sizes(nq, fmt):
    # group scales over all of E4M3 up to 64, zero among them, of either sign: products of scale and
    # code are exact, so nothing is lost but where a whole row is held against another
    g = _gen(15)
    n = 300
    kv, table = m4.cache(g, [n], 2, fmt, 32)
    codes = torch.tensor([c for c in range(256) if c & 127 <= 0x68], dtype=torch.uint8)
    for pool in (kv.k_group, kv.v_group):
        raw = pool.view(torch.uint8)
        new = codes[torch.randint(0, len(codes), raw.shape, generator=g)]
        raw.copy_(torch.where(raw.cpu() == 0x7F, raw.cpu(), new))
        pool.view(torch.uint8)[..., 0] = torch.where(raw.cpu()[..., 0] == 0x7F, raw.cpu()[..., 0], torch.tensor(0x68, dtype=torch.uint8)).cuda()
    Q = torch.randn((nq, 4, 128), generator=g).to(BF)
    _check(Q, kv, table, [n], [nq], True, 0)


SPANS = [  # queries, cached tokens, query heads, window, a key that only some queries see
    (5, 300, 2, 0, 297), (7, 900, 2, 300, 596), (140, 300, 1, 0, 200), (140, 2600, 1, 0, 2597), (140, 1200, 1, 500, 566),
]


def _span_case(nq, n, group, fmt):
    g = _gen(nq + n)
    kv, table = m4.cache(g, [n], 1, fmt, 32)
    return kv, table, torch.randn((nq, group, 128), generator=g).to(BF), torch.tensor([n], dtype=torch.int32).cuda()


def _check_rows(Q, kv, table, n, window, rows, out, lse=None, u_kv=0.0):
    K, V = m4.pool_rows(kv, "k", table[0], n)[0], m4.pool_rows(kv, "v", table[0], n)[0]
    spans = m4.seen(n, Q.shape[0], window)
    for hq in range(Q.shape[1]):
        want, want_lse, bound, lse_bound = m4.attend_rows(Q[:, hq].double().cpu(), K, V, rows, spans, out.dtype, u_kv)
        tp._within(out[list(rows), hq], want, bound, "head %d" % hq)
        if lse is not None:
            tp._within(lse[list(rows), hq], want_lse, lse_bound, "lse head %d" % hq)


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("nq,n,group,window,j", SPANS)
@pytest.mark.parametrize("which,size", [("v", math.inf), ("v", 2.0 ** 40), ("v", math.nan), ("k", 2.0 ** 40), ("k", math.nan)])
def test_scales_of_keys_that_some_queries_do_not_see(fmt, nq, n, group, window, j, which, size):
    kv, table, Q, lens = _span_case(nq, n, group, fmt)
    getattr(kv, which + "_scale")[int(table[0, j // 32]), 0, j % 32] = size
    out, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32, return_lse=True)
    alone = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window)
    sees = [i for i, (a, z) in enumerate(m4.seen(n, nq, window)) if a <= j < z]
    blind = [i for i in range(nq) if i not in sees]
    assert blind and sees
    rows = range(nq) if math.isfinite(size) and which == "v" else blind
    _check_rows(Q, kv, table, n, window, rows, out, lse)
    _check_rows(Q, kv, table, n, window, rows, alone, u_kv=0.0 if nq * group <= 16 else 2.0 ** -10)
    if not math.isfinite(size):
        assert not bool(out[sees].isfinite().any()) and not bool(alone[sees].isfinite().any())
        if which == "k":
            assert bool(lse[sees].isnan().all())


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("nq,n,group,window,j", SPANS + [(5, 15000, 8, 0, 14998)])
def test_nan_groups_of_keys_that_some_queries_do_not_see(fmt, nq, n, group, window, j):
    # page_write stores no NaN in a group's scale, but pages may come from elsewhere
    kv, table, Q, lens = _span_case(nq, n, group, fmt)
    page, row = int(table[0, j // 32]), j % 32
    kv.v_group.view(torch.uint8)[page, 0, row, 2] = 0x7F
    kv.v_group.view(torch.uint8)[page, 0, row, 7] = 0xFF
    out, lse = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32, return_lse=True)
    alone = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window)
    sees = [i for i, (a, z) in enumerate(m4.seen(n, nq, window)) if a <= j < z]
    blind = [i for i in range(nq) if i not in sees]
    assert blind and sees
    _check_rows(Q, kv, table, n, window, blind, out, lse)
    _check_rows(Q, kv, table, n, window, blind, alone, u_kv=0.0 if nq * group <= 16 else 2.0 ** -10)
    lost = list(range(32, 48)) + list(range(112, 128))
    keep = [c for c in range(128) if c not in lost]
    for o in (out, alone):
        assert bool(o[sees][..., lost].isnan().all()) and bool(o[sees][..., keep].isfinite().all())
    kv.k_group.view(torch.uint8)[page, 0, row, 0] = 0x7F
    out = api.page_attention(Q.cuda(), kv, table.cuda(), lens, window=window, out_dtype=F32)
    assert bool(out[sees].isnan().all())
    _check_rows(Q, kv, table, n, window, blind, out)


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("nq,n", [(3, 300), (140, 300), (140, 2600)])
def test_scores_far_past_the_exponential(fmt, nq, n):
    # as for 8-bit pages: a query's largest score has all the weight, and the output is its value
    kv, table, Q, lens = _span_case(nq, n, 2, fmt)
    scale = 3.0e8
    K, V = m4.pool_rows(kv, "k", table[0], n)[0], m4.pool_rows(kv, "v", table[0], n)[0]
    s = torch.einsum("ihd,jd->hij", Q.double(), K) * scale
    s = s.masked_fill(~(torch.arange(n)[None] <= torch.arange(n - nq, n)[:, None]), -math.inf)
    two = s.topk(2, -1).values
    clear = two[..., 0] - two[..., 1] > 128 * 2.0 ** -22 * (Q.double().abs().amax() * K.abs().amax() * 128 * scale)
    assert float(clear.double().mean()) > 0.5
    want = V[s.argmax(-1)]
    for kw in (dict(), dict(return_lse=True, out_dtype=F32)):
        out = api.page_attention(Q.cuda(), kv, table.cuda(), lens, scale=scale, **kw)
        out = out[0] if kw else out
        assert bool(out.isfinite().all())
        off = (out.double().cpu().transpose(0, 1) - want).abs()
        assert float(off[clear].max()) <= 3 * 2.0 ** -8 * float(V.abs().max())


@pytest.mark.parametrize("nq", [1, 50])
def test_bad_arguments_are_reported_on_the_device(nq):
    g = _gen(10)
    kv, table = m4.cache(g, [60, 60], 1, E2M1, 16)
    for t in (kv.k_scale, kv.v_scale):
        t.fill_(0.01)
    for t in (kv.k_group, kv.v_group):
        t.view(torch.uint8).fill_(0x50)
    lens = torch.tensor([60, 60], dtype=torch.int32).cuda()
    Q = torch.randn((2 * nq, 1, 128), generator=g).to(BF).cuda()
    good = api.page_attention(Q, kv, table.cuda(), lens)

    def status_of(table=table, lens=lens):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        return api.page_attention(Q, kv, table.cuda(), lens, status=st), int(st)
    assert status_of()[1] == 0
    for entry in (kv.n_pages, -1):
        bad = table.clone()
        bad[1, 1] = entry
        out, st = status_of(table=bad)
        assert st == qvg.QVG_DEV_BAD_INDEX and torch.equal(out[:nq], good[:nq])
    out, st = status_of(lens=torch.tensor([-4, 4000], dtype=torch.int32).cuda())
    assert st == qvg.QVG_DEV_BAD_INDEX and not out[:nq].any()


@pytest.mark.parametrize("nq,fmt", [(1, E2M1), (100, INT4)])
def test_capture_replay_other_streams_and_copied_handles(nq, fmt):
    import copy
    g = _gen(11)
    kv_lens = [900, 500]
    kv, table = m4.cache(g, kv_lens, 2, fmt, 64)
    table, lens = table.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
    freqs = api.rope_table(128)
    pos = torch.arange(2 * nq).cuda()
    slots = torch.stack([table[b, (kv_lens[b] - nq + torch.arange(nq).cuda()) // 64] * 64 +
                         (kv_lens[b] - nq + torch.arange(nq).cuda()) % 64 for b in range(2)]).flatten().long()
    x = torch.randn((2 * nq, 8, 128), generator=g).to(BF).cuda()

    def step(x, stream=None, kv=kv):
        q = api.rope(x[:, :4], pos, freqs, stream=stream)
        api.page_write(kv, x[:, 4:6], x[:, 6:], slots, rope=freqs, positions=pos, stream=stream)
        o = api.page_attention(q, kv, table, lens, stream=stream)
        return o, api.page_read(kv, table, lens, 900, stream=stream)
    want = [t.clone() for t in step(x)]
    assert all(torch.equal(a, b) for a, b in zip(step(x, kv=copy.deepcopy(kv)), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(x, side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = torch.randn(x.shape, generator=g).to(BF).cuda()
    buf = y.clone()
    with torch.cuda.stream(side):
        step(buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(buf)
    for src in (x, y, x):
        buf.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        ref = [t.clone() for t in step(src)]
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


@pytest.mark.parametrize("fmt", [E2M1, INT4])
def test_pages_can_be_copied_and_pickled(fmt):
    import copy
    import pickle
    kv, _ = m4.cache(_gen(3), [40], 2, fmt, 16)
    for other in (copy.deepcopy(kv), pickle.loads(pickle.dumps(kv))):
        assert other.k.dtype == fmt and other.k.data_ptr() != kv.k.data_ptr() and other.nbytes() == kv.nbytes()
        assert other.buffers().k == other.k.data_ptr() and other.buffers().v_group == other.v_group.data_ptr()
        for name in m4.POOLS:
            a, b = (getattr(x, name).view(torch.uint8) for x in (kv, other))
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("nq,seqs,n", [(1, 4, 15000), (5, 4, 15000), (1, 20, 3000), (300, 2, 4000)])
def test_calls_back_to_back(nq, seqs, n, fmt):
    # splits, shares and whole items launched one behind the other without a pause: every call the same
    g = _gen(nq + n)
    heads, page = 8, 64
    per = -(-n // page)
    kv = _blank(seqs * per, heads, page, fmt)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in (kv.k, kv.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=gen, device="cuda", dtype=torch.uint8) & 0x77)
    for t in (kv.k_group, kv.v_group):
        t.view(torch.uint8).copy_(torch.randint(0x40, 0x69, t.shape, generator=gen, device="cuda", dtype=torch.uint8))
    kv.k_scale.fill_(0.01)
    kv.v_scale.fill_(0.01)
    table = torch.randperm(seqs * per, generator=g).to(torch.int32).view(seqs, per).cuda()
    lens = torch.full((seqs,), n, dtype=torch.int32).cuda()
    Q = torch.randn((seqs * nq, 32 if nq < 100 else 8, 128), generator=g).to(BF).cuda()
    outs = [api.page_attention(Q, kv, table, lens, max_kv=n) for _ in range(60)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    assert bool(outs[0].float().abs().sum(-1).gt(0).all()) and bool(torch.isfinite(outs[0].float()).all())


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
def test_the_example_streams_through_4_bit_pages(fmt):
    # chunks written, attended to, read back and compressed: every chunk's attention against 64 bits
    import importlib.util
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("paged_stream4", os.path.join(root, "examples", "paged_stream.py"))
    example = importlib.util.module_from_spec(spec)
    sys.modules["paged_stream4"] = example
    spec.loader.exec_module(example)
    s = example.make_stream(heads=2, grid=(2, 6, 8), window=2, chunks=4, fmt=fmt, page=16, C=8)
    for k in range(4):
        Q, K, V = example.inputs(s, k, "cuda")
        pos = example.positions(s, "cpu")
        out = example.step(s, Q, K, V)
        assert s.packed == max(0, k - 2) and len(s.table) == min(k + 1, 3) * 6
        n = len(s.table) * 16
        tab = torch.tensor(s.table, dtype=torch.int32)
        Kp, Vp = m4.pool_rows(s.pages, "k", tab, n), m4.pool_rows(s.pages, "v", tab, n)
        Qr = api.rope(Q, pos.cuda(), s.rope).double().cpu()
        for h in range(2):
            want, _, bound, _ = pm.attend(Qr[:, h], Kp[h], Vp[h], 128 ** -0.5, False, 0, 2.0 ** -11, BF, 2.0 ** -10, 2.0 ** -10)
            tp._within(out[:, h], want, bound, "chunk %d head %d" % (k, h))


def test_offsets_past_32_bits():
    # rows past 2^32 bytes of codes: at the end of the pool, in 4 bits
    heads, page = 8, 128
    n_pages = (1 << 26) // (heads * page) + 4000      # 71 million rows of 64 bytes
    kv = api.allocate_pages(n_pages, heads, page, INT4)
    assert kv.k.numel() > 2 ** 32
    g = _gen(12)
    n, nq = 300, 70
    tab = torch.tensor([[n_pages - 1, n_pages - 3, 7]], dtype=torch.int32)
    i = torch.arange(n)
    K, V = (torch.randn((n, heads, 128), generator=g).to(BF).cuda() for _ in range(2))
    api.page_write(kv, K, V, (tab[0].long()[i // page] * page + i % page).cuda())
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    small = api.allocate_pages(3, heads, page, INT4)
    small_tab = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    api.page_write(small, K, V, (small_tab[0].long()[i // page] * page + i % page).cuda())
    assert torch.equal(api.page_read(kv, tab.cuda(), lens, n), api.page_read(small, small_tab.cuda(), lens, n))
    for q in (1, nq):
        Q = torch.randn((q, heads, 128), generator=g).to(BF).cuda()
        assert torch.equal(api.page_attention(Q, kv, tab.cuda(), lens, max_kv=n),
                           api.page_attention(Q, small, small_tab.cuda(), lens, max_kv=n))
