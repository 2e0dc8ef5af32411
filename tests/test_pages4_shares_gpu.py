"""GPU checks of attention of few rows over 4-bit pages in equal shares of all heads' keys, the form that
one token over many long sequences takes: the sizes where shares and stages nearly run out, and keys that
some queries do not see."""
import math

import pytest
import torch

from tests import pages4_model as m4
from tests import test_pages4_gpu as t4
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


def _wide(table, page, cells, rows):
    """The table with room for as many keys as equal shares want: four CTAs an SM up to eight rows, two for more."""
    ctas = 152 * (4 if rows <= 8 else 2)
    assert ctas // 4 < cells <= 2 * ctas
    longest = 1 + ctas * 2048 // cells
    wide = torch.zeros((table.shape[0], max(table.shape[1], -(-longest // page))), dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    return wide, longest, 2 * ctas * 16 * (128 + 2) * 4 + cells * 8


def _workspace(kv, n_seqs, q_heads, dtype, out_dtype, causal, window, total, most, max_pages, longest):
    return qvg.qvg_page_attention_workspace_bytes(qvg.qvg_page_attention_params(
        n_seqs=n_seqs, n_q_heads=q_heads, n_heads=kv.heads, d=128, page_tokens=kv.page_tokens, format=kv.format,
        q_dtype=api._DT[dtype], out_dtype=api._DT[out_dtype], n_pages=kv.n_pages, max_pages=max_pages, causal=int(causal),
        window=window, total_q=total, max_q=most, max_kv=longest, scale=0.1, q_token_stride=q_heads * 128,
        q_head_stride=128, o_token_stride=q_heads * 128, o_head_stride=128))


SHARES = [  # cached lengths, q lengths (in turn), q heads, heads, q type, format, page, causal, window
    ([2900, 0, 1, 64, 127, 128, 129, 700] * 3, [1], 16, 8, BF, E2M1, 64, True, 0),
    ([2900, 0, 1, 64, 127, 128, 129, 700] * 3, [1], 8, 8, HF, INT4, 128, False, 0),
    ([300, 900, 40, 2000], [1, 2], 96, 48, HF, INT4, 16, True, 250),   # a window that begins inside a share
    ([2000, 1500] * 2, [5], 40, 40, BF, E2M1, 32, True, 700),
    ([700, 4000, 33], [8], 60, 60, HF, INT4, 64, True, 900),
    ([17] * 11, [1], 16, 16, BF, INT4, 16, True, 0),                   # fewer stages than shares would like
    ([0, 0, 0, 0], [1, 0], 40, 40, BF, E2M1, 16, False, 0),            # no keys: a stage each where there is a query
    ([0, 0, 0, 0], [0, 0, 1, 0], 40, 40, HF, INT4, 16, False, 0),
    ([300, 20, 5], [0, 0, 1], 60, 60, BF, E2M1, 16, True, 0),          # a sequence with queries after two without
    ([128] * 304, [1], 2, 1, HF, INT4, 64, True, 0),                   # one stage a head
    ([129] * 152, [1], 4, 2, BF, E2M1, 32, True, 0),
    ([90] * 304, [1], 8, 4, BF, INT4, 16, True, 0),                    # as many heads as go in shares
    ([5, 3, 2500], [4], 60, 60, BF, INT4, 128, True, 0),               # some queries see nothing
    ([2000, 1500] * 2, [5], 60, 30, BF, INT4, 32, True, 700),          # nine to sixteen rows
    ([5, 3, 2500], [4], 90, 30, HF, E2M1, 128, True, 0),
]


@pytest.mark.parametrize("case", SHARES)
def test_equal_shares_of_4_bit_keys(case):
    # the workspace says that the call takes this way
    kv_lens, q_lens, q_heads, heads, dtype, fmt, page, causal, window = case
    q_lens = [q_lens[b % len(q_lens)] for b in range(len(kv_lens))]
    g = torch.Generator().manual_seed(sum(q_lens) + sum(kv_lens) + heads)
    kv, table = m4.cache(g, kv_lens, heads, fmt, page)
    wide, longest, bytes_ = _wide(table, page, heads * len(kv_lens), max(q_lens) * q_heads // heads)
    assert bytes_ == _workspace(kv, len(kv_lens), q_heads, dtype, dtype, causal, window, sum(q_lens), max(q_lens),
                                wide.shape[1], longest)
    Q = (1.5 * torch.randn((sum(q_lens), q_heads, 128), generator=g)).to(dtype)
    t4._check(Q, kv, wide, kv_lens, q_lens, causal, window, max_kv=longest)


@pytest.mark.parametrize("fmt", [E2M1, INT4])
@pytest.mark.parametrize("group", [1, 2])        # five and ten rows
@pytest.mark.parametrize("window", [0, 400])
def test_hidden_keys_in_equal_shares_of_4_bit_keys(fmt, group, window):
    # five queries over shares that end anywhere: a scale, and NaN group scales, of a key that only the last
    # two see
    g = torch.Generator().manual_seed(window + group)
    n, heads, nq = 1900, 80 // group, 5
    kv, table = m4.cache(g, [n, n], heads, fmt, 32)
    wide, longest, bytes_ = _wide(table, 32, 2 * heads, nq * group)
    Q = torch.randn((2 * nq, heads * group, 128), generator=g).to(BF)
    lens = torch.tensor([n, n], dtype=torch.int32).cuda()
    assert bytes_ == _workspace(kv, 2, heads * group, BF, F32, True, window, 2 * nq, nq, wide.shape[1], longest)

    def call():
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = api.page_attention(Q.cuda(), kv, wide.cuda(), lens, max_kv=longest, window=window, out_dtype=F32, return_lse=True,
                                 status=status)
        assert int(status) == 0
        return got
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
        was = kv.k_scale[page, :, row].clone()
        kv.k_scale[page, :, row] = size
        out, lse = call()
        assert torch.equal(out[:3], clean[:3]) and torch.equal(out[5:], clean[5:]) and torch.equal(lse[:3], clean_lse[:3])
        kv.k_scale[page, :, row] = was
    kv.v_group.view(torch.uint8)[page, :, row, 3] = 0x7F
    out, lse = call()
    # (rows done again: each is within its roundings, fp16 weights, of the same value)
    near = 8 * 2.0 ** -11 * float(m4.pool_rows(kv, "v", table[0], n - 2).abs().max())
    assert float((out[:3] - clean[:3]).abs().max()) <= near and torch.equal(out[5:], clean[5:])
    assert bool(out[3:5][..., 48:64].isnan().all()) and int(out.isnan().sum()) == 2 * heads * group * 16
    assert float((lse - clean_lse).abs().max()) <= 2.0 ** -12
    kv.k_group.view(torch.uint8)[page, :, row, 0] = 0xFF
    out, lse = call()
    assert float((out[:3] - clean[:3]).abs().max()) <= near and torch.equal(out[5:], clean[5:])
    assert bool(out[3:5].isnan().all()) and bool(lse[3:5].isnan().all())
