"""GPU checks of the paged-cache operators against their definitions in 64 bits
(pages_model.py), at the sizes, layouts and masks where they can go wrong.

Memory that no sequence reaches (rows past a length, pages of nobody) holds NaN in these tests,
and 8-bit scales there too.
"""
import math

import pytest
import torch

from tests import pages_model as pm
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


def _within(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s at %s: got %r want %r bound %r (%d off)" % (
            what, at, float(got[at]), float(want[at]), float(bound[at]), int(bad.sum())))


# ---------------------------------------------------------------- rotary positions

ROPE = [  # tokens, heads, dtype, rot, sections, interleaved, scaling, far, backward
    (1, 1, HF, 128, None, False, "none", 10, False),
    (3, 5, BF, 64, None, False, "by_parts", 2000000, False),
    (17, 9, F32, 8, None, True, "linear", 1000, True),
    (33, 12, BF, 128, (22, 21, 21), True, "none", 300, False),
    (130, 3, F32, 96, (20, 20, 4, 4), False, "stretched", 2 ** 31, False),
    (65, 8, HF, 120, None, True, "none", 70000, True),
    (9, 33, BF, 128, (0, 64), False, "none", 500, True),
]


@pytest.mark.parametrize("case", ROPE)
def test_rope(case):
    n, heads, dtype, rot, sections, inter, scaling, far, backward = case
    g = _gen(n)
    freqs, mscale = api.rope_frequencies(rot, sections=sections, scaling=scaling, factor=8.0)
    table = api.rope_table(rot, freqs=freqs, sections=sections, interleaved=inter, mscale=mscale)
    X = torch.randn((n, heads, 128), generator=g).to(dtype)
    pos = torch.randint(-far, far, (len(table.sections), n), generator=g)
    # far positions: the angle in the model, a double product, is off by 2^-53 of itself
    want, err = pm.rotate(X, pos, freqs.tolist(), table.sections, inter, mscale, backward)
    err = err + 2.0 ** -51 * far * X.double().abs().amax()
    bound = err + want.abs() * pm.HALF_EPS[dtype] + pm.TINY[dtype]
    got = api.rope(X.cuda(), pos.cuda(), table, backward=backward)
    _within(got, want, bound, "rope")
    assert torch.equal(got[..., rot:].cpu(), X[..., rot:])  # the rest is untouched


@pytest.mark.parametrize("far", [1, 3000, 2 ** 20])
def test_rope_angles_to_the_last_place(far):
    # sine and cosine within 3/4 of a step below 1 (2^-24), a product and a fused sum rounded by
    # at most 2^-24 each of |u| + |w|, and the angle cut to 2^-32 of a turn: 2.8 * 2^-24 in all
    g = _gen(far)
    freqs, _ = api.rope_frequencies(128)
    table = api.rope_table(128, freqs=freqs)
    X = torch.randn((2000, 2, 128), generator=g)
    pos = torch.randint(-far, far + 1, (1, 2000), generator=g)
    want, err = pm.rotate(X, pos, freqs.tolist(), table.sections, False)
    bound = err * (2.8 * 2.0 ** -24 / pm.ROTATE) + 2.0 ** -51 * far * X.double().abs().amax()
    _within(api.rope(X.cuda(), pos.cuda(), table), want, bound, "rope")


def test_rope_strides_in_place_and_broadcast():
    g = _gen(5)
    freqs, _ = api.rope_frequencies(64)
    table = api.rope_table(64, freqs=freqs)
    n, heads = 37, 6
    pos = torch.randint(0, 1000, (n,), generator=g).cuda()
    wide = torch.randn((n, 3 * heads, 128), generator=g).to(BF).cuda()
    X = wide[:, heads:2 * heads]  # rows of a fused projection
    plain = api.rope(X.contiguous(), pos, table)
    assert torch.equal(api.rope(X, pos, table), plain)
    heads_first = X.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((heads, n, 128), dtype=BF, device="cuda").transpose(0, 1)
    assert api.rope(heads_first, pos, table, out=out) is out and torch.equal(out, plain)
    before = wide.clone()
    api.rope(X, pos, table, out=X)
    assert torch.equal(X, plain)
    assert torch.equal(wide[:, :heads], before[:, :heads])
    assert torch.equal(wide[:, 2 * heads:], before[:, 2 * heads:])
    one = torch.randn((n, 1, 128), generator=g).to(BF).cuda()
    assert torch.equal(api.rope(one.expand(n, heads, 128), pos, table),
                       api.rope(one.expand(n, heads, 128).contiguous(), pos, table))
    assert api.rope(X[:0], pos[:0], table).shape == (0, heads, 128)


def test_rope_backward_is_the_gradient():
    # against the formula's transpose and against differences (the map is linear: exact)
    g = _gen(6)
    freqs, mscale = api.rope_frequencies(32, scaling="by_parts", factor=4.0)
    table = api.rope_table(32, freqs=freqs, mscale=mscale)
    x, dy = (torch.randn((4, 2, 128), generator=g).cuda() for _ in range(2))
    e = torch.randn((4, 2, 128), generator=g).cuda()
    pos = torch.randint(0, 5000, (4,), generator=g).cuda()
    dx = api.rope(dy, pos, table, backward=True)
    change = api.rope(x + e, pos, table).double() - api.rope(x, pos, table).double()
    a, b = float((change * dy.double()).sum()), float((dx.double() * e.double()).sum())
    size = float((e.abs() * dy.abs()).sum() + 4 * (x.abs() * dy.abs()).sum())
    assert abs(a - b) <= 4 * pm.ROTATE * size * 2


# ---------------------------------------------------------------- the pages

def _written(case_seed, n, heads, dtype, fmt, page, table=None, pos=None, strided=False):
    g = _gen(case_seed)
    rows = torch.randn((n, 2 * heads, 128), generator=g)
    rows[..., 3::50] += 30.0
    rows = rows.to(dtype)
    K, V = rows[:, :heads], rows[:, heads:]
    pages = -(-n // page) + 3
    kv = api.allocate_pages(pages, heads, page, fmt)
    for t in (kv.k, kv.v):
        t.view(torch.uint8).fill_(0)
    for t in (kv.k_scale, kv.v_scale):
        if t is not None:
            t.fill_(-1.0)
    order = torch.randperm(pages, generator=g)
    i = torch.arange(n)
    slots = order[i // page] * page + i % page
    return rows, K, V, kv, order, slots


WRITE = [  # tokens, heads, dtype, format, page, rotary part (0: none), interleaved
    (1, 1, BF, E4, 16, 128, False),
    (5, 3, HF, I8, 16, 0, False),
    (67, 7, F32, E4, 32, 0, False),
    (67, 12, BF, BF, 64, 128, True),
    (131, 4, F32, HF, 128, 64, False),
    (40, 5, HF, HF, 64, 0, False),
    (129, 9, BF, I8, 128, 96, False),
    (33, 2, F32, I8, 32, 0, False),
    (20, 6, HF, E4, 16, 32, True),
    (11, 4, F32, BF, 16, 0, False),
]


@pytest.mark.parametrize("case", WRITE)
def test_page_write_and_read(case):
    n, heads, dtype, fmt, page, rot, inter = case
    rows, K, V, kv, order, slots = _written(n, n, heads, dtype, fmt, page)
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
    for name, x64, err in (("k", want_k, err_k), ("v", V.double(), torch.zeros_like(err_k))):
        pool, scale = getattr(kv, name), getattr(kv, name + "_scale")
        flat = pool.transpose(1, 2).flatten(0, 1).cpu()  # [slot][heads][128]
        got = pm.take(flat, slots)
        if scale is None:
            _within(got, x64, err + x64.abs() * pm.HALF_EPS[fmt] + pm.TINY[fmt], name)
        else:
            s = scale.transpose(1, 2).flatten(0, 1).cpu()[slots]
            amax = x64.abs().amax(-1)
            # the scale: one rounding of a quotient of a largest magnitude known to err
            _within(s, amax / pm.TOP[fmt], (amax * 2.0 ** -23 + err.amax(-1)) / pm.TOP[fmt], "scale")
            y = got.double() * s.double()[..., None]
            # half a step: of 1 for int8; of 2^-3 of the binade, or 2^-9, for e4m3; the quotient
            # before rounding carries two roundings of 2^-24 and the scale one
            step = torch.ones_like(y) if fmt == I8 else torch.exp2(
                torch.floor(torch.log2((x64.abs() / (amax / pm.TOP[fmt])[..., None]).clamp(min=2.0 ** -6))) - 3)
            half = step * (amax / pm.TOP[fmt])[..., None] / 2
            _within(y, x64, half * (1 + 2.0 ** -7) + 2 * err + amax[..., None] * 2.0 ** -21, name)
            if not (rot and name == "k"):  # and exactly, where the input is exact
                codes, want_s = pm.stored((K if name == "k" else V).float(), fmt)
                assert torch.equal(got.view(torch.uint8), codes.view(torch.uint8))
                assert torch.equal(s, want_s)
            rest = torch.ones(scale.numel() // heads, dtype=torch.bool)
            rest[slots] = False
            assert bool((scale.transpose(1, 2).flatten(0, 1).cpu()[rest] == -1.0).all())
        rest = torch.ones(flat.shape[0], dtype=torch.bool)
        rest[slots] = False
        assert not flat.view(torch.uint8)[rest].any()  # no other row was touched
    # read back: whole, and a part that begins and ends inside pages
    tab = torch.full((2, kv.n_pages), -7, dtype=torch.int32)
    tab[0, :-(-n // page)] = order[:-(-n // page)].to(torch.int32)
    lens = torch.tensor([n, 0], dtype=torch.int32).cuda()
    for out_dtype in (BF, HF, F32):
        for first, count in ((0, n), (n // 3, n), (n, 5)):
            X = api.page_read(kv, tab.cuda(), lens, count, first=first, out_dtype=out_dtype, status=status)
            assert X.shape == (2, 2 * heads, count, 128)
            for which, name in enumerate(("k", "v")):
                want = pm.pool_rows(getattr(kv, name), getattr(kv, name + "_scale"), tab[0], n, page)[:, first:first + count]
                have = want.shape[1]
                bound = want.abs() * (pm.HALF_EPS[out_dtype] + 2.0 ** -23) + pm.TINY[out_dtype]
                _within(X[0, which::2, :have], want, bound, "read")
                assert not X[0, which::2, have:].any() and not X[1].any()
    assert int(status) == 0


def test_page_write_skips_and_reports():
    heads, page = 3, 16
    kv = api.allocate_pages(4, heads, page, E4)
    for t in (kv.k, kv.v):
        t.view(torch.uint8).fill_(0)
    kv.k_scale.fill_(-1.0)
    kv.v_scale.fill_(-1.0)
    K = torch.randn((5, heads, 128), generator=_gen(2)).cuda()
    V = torch.randn((5, heads, 128), generator=_gen(3)).cuda()
    K[1, 0, 7] = float("nan")
    V[2, 2, 0] = float("-inf")
    K[3, 1] = 0.0
    V[3, 1] = 2.0 ** -101
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.page_write(kv, K, V, torch.tensor([-1, 17, 18, 19, 4 * page]).cuda(), status=status)
    assert int(status) == qvg.QVG_DEV_NONFINITE | qvg.QVG_DEV_BAD_INDEX
    ks, vs = kv.k_scale.cpu(), kv.v_scale.cpu()
    assert int((ks == -1).sum()) == int((vs == -1).sum()) == (4 * page - 3) * heads
    assert bool(ks[1, 0, 1].isnan()) and bool(vs[1, 2, 2].isnan())
    assert int(ks.isnan().sum()) == int(vs.isnan().sum()) == 1
    assert ks[1, 1, 3] == 0 and vs[1, 1, 3] == 0 and not kv.v[1, 1, 3].view(torch.uint8).any()
    # such a row reads as NaN, and only it
    tab = torch.tensor([[1]], dtype=torch.int32).cuda()
    X = api.page_read(kv, tab, torch.tensor([4], dtype=torch.int32).cuda(), 4)
    assert bool(X[0, 0, 1].isnan().all()) and bool(X[0, 5, 2].isnan().all())
    assert int(X.isnan().sum()) == 2 * 128
    status.zero_()
    api.page_write(kv, K[:0], V[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), status=status)
    assert int(status) == 0


def test_page_read_bad_table_and_strides():
    kv = api.allocate_pages(3, 2, 16, BF)
    kv.k.fill_(1.0)
    kv.v.fill_(2.0)
    tab = torch.tensor([[2, 9], [-3, 1]], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    X = api.page_read(kv, tab, torch.tensor([20, 99], dtype=torch.int32).cuda(), 40, status=status)
    assert int(status) == qvg.QVG_DEV_BAD_INDEX
    assert bool((X[0, 0, :16] == 1).all()) and not X[0, :, 16:].any()   # entry 9 is outside
    assert not X[1, :, :16].any() and bool((X[1, 1, 16:32] == 2).all())  # cut to the table
    assert not X[1, :, 32:].any()
    big = torch.full((2, 6, 50, 128), 5.0, dtype=torch.float32, device="cuda")
    part = big[:, 1:5, 3:33]
    api.page_read(kv, tab, torch.tensor([16, 0], dtype=torch.int32).cuda(), 30, out=part)
    assert bool((part[0, 2, :16] == 1).all()) and not part[0, 0, 16:].any() and not part[1].any()
    part.fill_(5.0)
    assert bool((big == 5).all())


# ---------------------------------------------------------------- attention

def _cache(g, kv_lens, heads, fmt, page, hidden_values=None):
    need = [-(-n // page) for n in kv_lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(kv_lens), max(1, max(need)) + 1), -5, dtype=torch.int32)
    written = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k].to(torch.int32)
        rows = torch.arange(k * page) < kv_lens[b]
        written[order[at:at + k]] = rows.view(k, page)
        at += k
    pools = {}
    for name in ("k", "v"):
        x = torch.randn((pages, heads, page, 128), generator=g)
        if fmt in pm.TOP:
            codes, scale = pm.stored(x, fmt)
            pools[name] = torch.where(written[:, None, :, None], codes.view(torch.uint8), torch.tensor(0x7F, dtype=torch.uint8)).view(fmt)
            pools[name + "_scale"] = torch.where(written[:, None], scale, torch.tensor(math.nan))
        else:
            pools[name] = torch.where(written[:, None, :, None], x, torch.tensor(math.nan)).to(fmt)
            pools[name + "_scale"] = None
    kv = api.PagedKV(*(None if pools[x] is None else pools[x].cuda() for x in ("k", "v", "k_scale", "v_scale")))
    return kv, table


def _check(Q, kv, table, kv_lens, q_lens, causal, window, scale=None, out=None, out_dtype=None, **kw):
    heads, page, group = kv.heads, kv.page_tokens, Q.shape[1] // kv.heads
    cu = torch.tensor([sum(q_lens[:b]) for b in range(len(q_lens) + 1)], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(dict(cu_q=cu.cuda(), max_q=max(q_lens), max_kv=max(kv_lens)), **kw)
    got, lse = api.page_attention(Q.cuda() if not Q.is_cuda else Q, kv, table.cuda(),
                                  torch.tensor(kv_lens, dtype=torch.int32).cuda(), causal=causal,
                                  window=window, scale=scale, out=out, out_dtype=out_dtype, return_lse=True,
                                  status=status, **kw)
    # without the log-sum-exp and with a bf16 output: 8-bit keys and values may meet many rows
    # rounded to fp16
    alone = api.page_attention(Q.cuda() if not Q.is_cuda else Q, kv, table.cuda(),
                               torch.tensor(kv_lens, dtype=torch.int32).cuda(), causal=causal,
                               window=window, scale=scale, out_dtype=got.dtype, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    narrow = kv.k.dtype in pm.TOP
    u_p = pm.HALF_EPS[HF if narrow else Q.dtype]
    u_kv = pm.HALF_EPS[HF] if narrow and got.dtype is BF and max(q_lens) * group > 16 else 0.0
    if not u_kv:
        assert torch.equal(alone, got)
    Qc = Q.double().cpu()
    for b, (nq, n) in enumerate(zip(q_lens, kv_lens)):
        if nq == 0:
            continue
        K = pm.pool_rows(kv.k, kv.k_scale, table[b], n, page)
        V = pm.pool_rows(kv.v, kv.v_scale, table[b], n, page)
        rows = slice(int(cu[b]), int(cu[b]) + nq)
        for hq in range(Q.shape[1]):
            want, want_lse, bound, lse_bound = pm.attend(
                Qc[rows, hq], K[hq // group], V[hq // group], 128 ** -0.5 if scale is None else scale,
                causal, window, u_p, got.dtype)
            _within(got[rows, hq], want, bound, "sequence %d head %d" % (b, hq))
            if u_kv:
                _, _, wider, _ = pm.attend(
                    Qc[rows, hq], K[hq // group], V[hq // group], 128 ** -0.5 if scale is None else scale,
                    causal, window, u_p, got.dtype, u_kv, u_kv)
                _within(alone[rows, hq], want, wider, "alone: sequence %d head %d" % (b, hq))
            none = want_lse == -math.inf
            assert torch.equal(lse[rows, hq].cpu() == -math.inf, none)
            _within(lse[rows, hq].cpu()[~none], want_lse[~none], lse_bound[~none], "lse")
    return got, lse


ATTEND = [  # q lengths, cached lengths, q heads, heads, q type, format, page, causal, window
    ([1], [1], 1, 1, BF, BF, 16, True, 0),
    ([1, 1, 1], [5, 0, 300], 8, 2, BF, BF, 16, True, 0),      # an empty sequence sees nothing
    ([1] * 4, [33, 64, 1000, 127], 4, 4, HF, HF, 32, True, 0),
    ([1, 1], [4000, 517], 16, 2, BF, E4, 64, True, 0),          # splits
    ([1, 1], [3900, 40], 7, 1, HF, I8, 128, True, 700),
    ([3, 5, 2], [3, 200, 77], 4, 2, HF, E4, 16, True, 0),
    ([4, 2], [2, 90], 3, 3, BF, BF, 16, True, 0),               # first rows see nothing
    ([2, 0, 7], [900, 10, 450], 6, 2, BF, I8, 32, False, 0),
    ([70], [70], 2, 2, BF, BF, 64, True, 0),
    ([129, 17], [513, 17], 4, 1, HF, HF, 16, True, 100),
    ([200], [391], 2, 2, BF, BF, 128, False, 0),
    ([300, 1, 45], [300, 700, 1000], 8, 4, BF, E4, 32, True, 0),
    ([260], [1300], 3, 1, HF, I8, 64, False, 0),
    ([150], [1200], 2, 1, HF, E4, 64, True, 64),
    ([257], [257], 1, 1, BF, I8, 16, False, 33),                # a window without causality
    ([64], [3000], 1, 1, BF, BF, 64, True, 0),                  # many splits of one tile
    ([31], [31], 128, 1, BF, BF, 16, True, 0),                  # 128 query heads share one
    ([513], [640], 5, 5, HF, HF, 128, True, 0),
    ([257], [1100], 77, 77, BF, BF, 64, True, 0),               # more than a round: whole items, split ones
    ([40, 20], [2500, 900], 2, 2, HF, I8, 16, True, 0),         # few items of unlike sequences: all split
    ([2], [5000], 8, 1, BF, E4, 128, True, 3000),               # 16 rows, splits through memory
]


@pytest.mark.parametrize("case", ATTEND)
def test_page_attention(case):
    q_lens, kv_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    g = _gen(sum(q_lens) + sum(kv_lens))
    kv, table = _cache(g, kv_lens, heads, fmt, page)
    Q = (1.5 * torch.randn((sum(q_lens), q_heads, 128), generator=g)).to(dtype)
    _check(Q, kv, table, kv_lens, q_lens, causal, window)


RAGGED = [  # as ATTEND: more items than SMs, those that see the most first
    ([300, 0, 70, 513], [400, 50, 70, 1200], 44, 44, BF, BF, 32, True, 0),
    ([40, 260], [41, 700], 90, 90, HF, I8, 16, True, 300),
    ([33, 1, 0, 257, 257], [20, 0, 9, 300, 300], 40, 40, BF, E4, 64, False, 0),
]


@pytest.mark.parametrize("case", RAGGED)
def test_page_attention_of_many_heads_and_unlike_sequences(case):
    q_lens, kv_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    g = _gen(sum(q_lens) + heads)
    kv, table = _cache(g, kv_lens, heads, fmt, page)
    Q = torch.randn((sum(q_lens), q_heads, 128), generator=g).to(dtype)
    _check(Q, kv, table, kv_lens, q_lens, causal, window)


SHARES = [  # longest and other cached lengths, q lengths, q heads, heads, q type, format, page, causal, window
    ([2900, 0, 1, 64, 127, 128, 129, 700] * 3, [1], 8, 4, BF, BF, 64, True, 0),
    ([1500, 0, 1, 64, 127, 128, 129, 700] * 3, [2, 0, 1, 3], 10, 5, BF, I8, 32, True, 0),
    ([5, 3, 2500], [4], 90, 30, HF, E4, 128, True, 0),           # 12 rows; some see nothing
    ([300, 900, 40, 2000], [1, 2], 48, 24, HF, HF, 16, True, 250),
    ([1000, 10, 333], [5, 1], 27, 27, BF, E4, 64, False, 0),
    ([17] * 11, [1], 8, 8, BF, BF, 16, True, 0),                 # a share each, and none to spare
    ([1, 0, 2], [1], 40, 40, HF, I8, 16, True, 0),
    ([0, 0, 0, 0], [1, 0], 20, 20, BF, BF, 16, False, 0),
    ([600] * 40, [1], 8, 8, BF, I8, 16, True, 0),
]


@pytest.mark.parametrize("case", SHARES)
def test_page_attention_in_equal_shares(case):
    # many heads of sequences that may be long, as far as the call can know: their keys are cut
    # into equal shares, wherever a head ends
    kv_lens, q_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    q_lens = [q_lens[b % len(q_lens)] for b in range(len(kv_lens))]
    g = _gen(sum(q_lens) + sum(kv_lens) + heads)
    kv, table = _cache(g, kv_lens, heads, fmt, page)
    longest = 1 + 152 * 2 * 2048 // (heads * len(kv_lens))
    wide = torch.zeros((len(kv_lens), max(table.shape[1], -(-longest // page))), dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    Q = (1.5 * torch.randn((sum(q_lens), q_heads, 128), generator=g)).to(dtype)
    _check(Q, kv, wide, kv_lens, q_lens, causal, window, max_kv=longest)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("nq", [1, 40])
def test_page_attention_lengths(n, nq):
    nq = min(n, nq)
    g = _gen(1000 + n)
    kv, table = _cache(g, [n], 1, BF, 16)
    Q = torch.randn((nq, 3, 128), generator=g).to(BF)
    _check(Q, kv, table, [n], [nq], True, 0)
    _check(Q, kv, table, [n], [nq], False, 0)


@pytest.mark.parametrize("nq,n,fmt", [(1, 700, BF), (90, 500, BF), (90, 500, E4)])
def test_page_attention_large_scores(nq, n, fmt):
    # scores of several hundred, rising and falling along the keys: the running maximum moves
    g = _gen(77)
    kv, table = _cache(g, [n], 1, fmt, 32)
    ramp = torch.linspace(-40, 40, kv.n_pages * 32)[torch.randperm(kv.n_pages * 32, generator=g)]
    if fmt is BF:
        kv.k.copy_((kv.k.float().cpu() + ramp.view(kv.n_pages, 1, 32, 1)).to(BF))
    Q = (3 * torch.randn((nq, 2, 128), generator=g) + 0.3).to(BF)
    _check(Q, kv, table, [n], [nq], True, 0)


def test_page_attention_strides_types_and_default_arguments():
    g = _gen(8)
    kv_lens, q_lens = [50, 300], [20, 20]
    kv, table = _cache(g, kv_lens, 2, HF, 32)
    wide = torch.randn((40, 12, 128), generator=g).to(HF).cuda()
    Q = wide[:, 2:6]
    plain, lse = _check(Q, kv, table, kv_lens, q_lens, True, 0)
    for out_dtype in (BF, F32, HF):
        out = torch.zeros((4, 40, 128), dtype=out_dtype, device="cuda").transpose(0, 1)
        _check(Q, kv, table, kv_lens, q_lens, True, 0, out=out)
    lens = torch.tensor(kv_lens, dtype=torch.int32).cuda()
    again = api.page_attention(Q, kv, table.cuda(), lens)  # equal shares, no bounds given
    assert again.shape == plain.shape
    _check(Q, kv, table, kv_lens, q_lens, True, 0, max_kv=None, max_q=None)
    _check(Q, kv, table, kv_lens, q_lens, True, 0, scale=-0.3)
    one = torch.randn((40, 1, 128), generator=g).to(HF).cuda().expand(40, 4, 128)
    _check(one, kv, table, kv_lens, q_lens, True, 0)
    _check(Q, kv, table, kv_lens, q_lens, True, 0, scale=0.0)


@pytest.mark.parametrize("nq", [1, 60])
def test_value_scales_of_many_sizes(nq):
    # value scales from 2^-60 to 2^60, rising, falling and mixed along the keys, so that the
    # reference they are held against has to move; the weights are large where scales are small
    g = _gen(14)
    n, page = 700, 16
    for order in ("rising", "falling", "mixed"):
        kv, table = _cache(g, [n], 1, E4, page)
        e = torch.linspace(-60, 60, n) * (-1 if order == "falling" else 1)
        if order == "mixed":
            e = e[torch.randperm(n, generator=g)]
        for j in range(n):
            kv.v_scale[int(table[0, j // page]), 0, j % page] = 2.0 ** float(e[j])
        Q = torch.randn((nq, 2, 128), generator=g).to(HF)
        _check(Q, kv, table, [n], [nq], True, 0, out_dtype=F32)  # past fp16's largest number


@pytest.mark.parametrize("fmt", [BF, I8])
@pytest.mark.parametrize("nq,n,group", [(5, 300, 2), (140, 300, 1), (140, 2600, 1)])
def test_what_a_query_does_not_see_cannot_change_it(fmt, nq, n, group):
    # NaN and infinities in a late key and value: earlier queries' rows stay as they were, later
    # ones are NaN or infinite, channel by channel, as the formula says
    g = _gen(9)
    kv, table = _cache(g, [n], 1, fmt, 32)
    Q = torch.randn((nq, group, 128), generator=g).to(BF)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    clean = api.page_attention(Q.cuda(), kv, table.cuda(), lens)
    j = n - 3  # seen by the last three queries
    page, row = int(table[0, j // 32]), j % 32
    if fmt is BF:
        kv.v[page, 0, row, 5] = float("inf")
        kv.v[page, 0, row, 9] = float("nan")
    else:
        kv.v_scale[page, 0, row] = float("nan")
    got = api.page_attention(Q.cuda(), kv, table.cuda(), lens)
    assert bool(got[:-3].isfinite().all())
    # (a row computed once more has unrounded weights: each side is within its roundings, half a
    # bf16 step of every weight and of the result, of the same value)
    near = 4 * 2.0 ** -8 * float(pm.pool_rows(kv.v, kv.v_scale, table[0], n - 3, 32).abs().max())
    assert float((got[:-3].float() - clean[:-3].float()).abs().max()) <= (near if fmt is BF else 0.0)
    if fmt is BF:
        assert bool((got[-3:, :, 5] == float("inf")).all()) and bool(got[-3:, :, 9].isnan().all())
        keep = [c for c in range(128) if c not in (5, 9)]
        err = (got[-3:, :, keep].float() - clean[-3:, :, keep].float()).abs()
        assert float(err.max()) <= near
    else:
        assert bool(got[-3:].isnan().all())
    kv.v_scale is None or kv.v_scale[page, 0, row].fill_(0.1)
    kv.k[page, 0, row, 0] = float("nan") if fmt is BF else 0
    if fmt is BF:
        kv.v[page, 0, row] = 0.0
        got = api.page_attention(Q.cuda(), kv, table.cuda(), lens)
        assert float((got[:-3].float() - clean[:-3].float()).abs().max()) <= near
        assert bool(got[-3:].isnan().all())


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("size", [0.0, 1e-30, 1e30])
def test_queries_and_keys_of_extreme_sizes(fmt, size):
    # rows of zeros in the cache (scale 0), queries whose products with anything vanish
    g = _gen(15)
    n, nq = 200, 60
    kv, table = _cache(g, [n], 1, fmt, 32)
    for j in range(0, n, 2) if size else range(n):
        page, row = int(table[0, j // 32]), j % 32
        kv.k[page, 0, row].view(torch.uint8).zero_()
        if kv.k_scale is not None:
            kv.k_scale[page, 0, row] = 0.0
    Q = (torch.randn((nq, 2, 128), generator=g) * (size or 1e-30)).to(BF)
    scale = 1e-31 if size > 1 else 0.1
    _check(Q, kv, table, [n], [nq], True, 0, scale=scale)
    _check(Q[:4], kv, table, [n], [4], True, 0, scale=scale)


def test_page_attention_reports_bad_arguments_on_the_device():
    g = _gen(10)
    kv, table = _cache(g, [60, 60], 1, BF, 16)
    kv.k.copy_(torch.randn(kv.k.shape, generator=g))
    kv.v.copy_(torch.randn(kv.v.shape, generator=g))
    lens = torch.tensor([60, 60], dtype=torch.int32).cuda()
    for nq in (1, 50):  # both kernels
        Q = torch.randn((2 * nq, 1, 128), generator=g).to(BF).cuda()
        good = api.page_attention(Q, kv, table.cuda(), lens)

        def status_of(table=table, lens=lens, cu=None, max_q=None):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.full_like(Q, 7.0)
            api.page_attention(Q, kv, table.cuda(), lens, cu_q=cu, max_q=max_q, status=st, out=out)
            return int(st), out
        assert status_of()[0] == 0
        bad = table.clone()
        bad[1, 1] = kv.n_pages
        st, out = status_of(table=bad)
        assert st == qvg.QVG_DEV_BAD_INDEX and torch.equal(out[:nq], good[:nq])
        bad[1, 1] = -1
        assert status_of(table=bad)[0] == qvg.QVG_DEV_BAD_INDEX
        st, out = status_of(lens=torch.tensor([60, 4000], dtype=torch.int32).cuda())
        assert st == qvg.QVG_DEV_BAD_INDEX and torch.equal(out[:nq], good[:nq])
        st, out = status_of(lens=torch.tensor([-4, 60], dtype=torch.int32).cuda())
        assert st == qvg.QVG_DEV_BAD_INDEX and not out[:nq].any() and torch.equal(out[nq:], good[nq:])
        for cu in ([0, nq, 2 * nq + 9], [0, -3, 2 * nq], [nq, 0, nq]):
            st, out = status_of(cu=torch.tensor(cu, dtype=torch.int32).cuda(), max_q=2 * nq)
            assert st == qvg.QVG_DEV_BAD_INDEX
        # more queries than max_q allows: the rows left out are not written
        st, out = status_of(cu=torch.tensor([0, 0, 2 * nq], dtype=torch.int32).cuda(), max_q=2 * nq - 1)
        assert st == qvg.QVG_DEV_BAD_INDEX and bool((out[-1] == 7).all())
        assert not bool((out[:-1] == 7).all(-1).any())


@pytest.mark.parametrize("nq,heads,fmt", [(1, 90, I8), (300, 90, BF)])
def test_many_heads_report_bad_arguments_on_the_device(nq, heads, fmt):
    # equal shares, and items in the order of what they see: what is bad is reported all the same
    g = _gen(12)
    kv, table = _cache(g, [300, 0], heads, fmt, 16)
    table = torch.cat([table, torch.zeros((2, 300), dtype=torch.int32)], 1)
    total = nq + 1
    Q = torch.randn((total, heads, 128), generator=g).to(BF).cuda()

    def status_of(table=table, lens=(300, 0), cu=(0, nq, total)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(Q, 7.0)
        api.page_attention(Q, kv, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           cu_q=torch.tensor(cu, dtype=torch.int32).cuda(), max_q=nq, status=st, out=out)
        return int(st), out
    st, good = status_of()
    assert st == 0 and not good[nq:].any() and not bool((good == 7).all(-1).any())
    bad = table.clone()
    bad[0, 3] = kv.n_pages
    assert status_of(table=bad)[0] == qvg.QVG_DEV_BAD_INDEX
    bad[0, 3] = -1
    assert status_of(table=bad)[0] == qvg.QVG_DEV_BAD_INDEX
    st, out = status_of(lens=(300, -5))
    assert st == qvg.QVG_DEV_BAD_INDEX and torch.equal(out, good)
    assert status_of(lens=(table.shape[1] * 16 + 1, 0))[0] == qvg.QVG_DEV_BAD_INDEX
    for cu in ((0, nq, total + 9), (0, -3, nq), (nq, 0, nq)):
        assert status_of(cu=cu)[0] == qvg.QVG_DEV_BAD_INDEX


@pytest.mark.parametrize("nq", [1, 100])
def test_capture_replay_and_other_streams(nq):
    g = _gen(11)
    kv_lens = [900, 500]
    kv, table = _cache(g, kv_lens, 2, E4, 64)
    table, lens = table.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
    freqs = api.rope_table(128)
    pos = torch.arange(2 * nq).cuda()
    slots = torch.stack([table[b, (kv_lens[b] - nq + torch.arange(nq).cuda()) // 64] * 64 +
                         (kv_lens[b] - nq + torch.arange(nq).cuda()) % 64 for b in range(2)]).flatten().long()
    x = torch.randn((2 * nq, 8, 128), generator=g).to(BF).cuda()

    def step(x, stream=None):
        q = api.rope(x[:, :4], pos, freqs, stream=stream)
        api.page_write(kv, x[:, 4:6], x[:, 6:], slots, rope=freqs, positions=pos, stream=stream)
        o = api.page_attention(q, kv, table, lens, stream=stream)
        return o, api.page_read(kv, table, lens, 900, stream=stream)
    want = [t.clone() for t in step(x)]
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


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("nq", [1, 5])
def test_split_calls_back_to_back(nq, fmt):
    # long sequences in parts, launched one behind the other without a pause: every call the same
    g = _gen(nq)
    n, heads, page, seqs = 15000, 8, 64, 4
    per = -(-n // page)
    kv = api.allocate_pages(seqs * per, heads, page, fmt)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in (kv.k, kv.v):
        t.copy_((torch.randn(t.shape, generator=gen, device="cuda") * (1 if kv.k_scale is None else 60)).clamp(-127, 127).to(fmt))
    if kv.k_scale is not None:
        kv.k_scale.fill_(0.02)
        kv.v_scale.fill_(0.02)
    table = torch.randperm(seqs * per, generator=g).to(torch.int32).view(seqs, per).cuda()
    lens = torch.full((seqs,), n, dtype=torch.int32).cuda()
    Q = torch.randn((seqs * nq, 32, 128), generator=g).to(BF).cuda()
    outs = [api.page_attention(Q, kv, table, lens, max_kv=n) for _ in range(60)]
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    assert bool(outs[0].float().abs().sum(-1).gt(0).all()) and bool(torch.isfinite(outs[0].float()).all())


def test_offsets_past_32_bits():
    # a pool of 2^31 + bytes per array: rows at its end, in 16 bits
    heads, page = 8, 128
    n_pages = (1 << 23) // (heads * page) + 40        # 8.4 million rows of 256 bytes
    kv = api.allocate_pages(n_pages, heads, page, BF)
    assert kv.k.numel() > 2 ** 30
    g = _gen(12)
    n, nq = 300, 70
    tab = torch.tensor([[n_pages - 1, n_pages - 3, 7]], dtype=torch.int32)
    i = torch.arange(n)
    slots = (tab[0].long()[i // page] * page + i % page).cuda()
    K, V = (torch.randn((n, heads, 128), generator=g).to(BF).cuda() for _ in range(2))
    api.page_write(kv, K, V, slots)
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    X = api.page_read(kv, tab.cuda(), lens, n)
    assert torch.equal(X[0, 0::2].transpose(0, 1), K) and torch.equal(X[0, 1::2].transpose(0, 1), V)
    small = api.allocate_pages(3, heads, page, BF)
    small_tab = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    api.page_write(small, K, V, (small_tab[0].long()[i // page] * page + i % page).cuda())
    for q in (1, nq):
        Q = torch.randn((q, heads, 128), generator=g).to(BF).cuda()
        assert torch.equal(api.page_attention(Q, kv, tab.cuda(), lens),
                           api.page_attention(Q, small, small_tab.cuda(), lens))
