"""What the paged-cache calls refuse without a GPU in the machine."""
import pytest
import torch

from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg


def test_host_tensors_are_refused_by_every_call():
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    lens, table = torch.zeros(1, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    kv = type("Pages", (), dict(k=x, heads=2, gpu=-1))()
    with pytest.raises(ValueError):
        api.page_attention(x, kv, table, lens)
    with pytest.raises(ValueError):
        api.page_write(kv, x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        api.page_read(kv, table, lens, 4)
    with pytest.raises(ValueError):
        api.rope(x, torch.zeros(4, dtype=torch.int64), None)
    with pytest.raises(ValueError):
        api.allocate_pages(2, 1, 16, torch.bfloat16, device="cpu")
    with pytest.raises(ValueError):
        api.rope_table(64, device="cpu")


@pytest.mark.parametrize("bad", [dict(fast_turns=1.0), dict(fast_turns=2.0, slow_turns=2.0), dict(fast_turns=1.0, slow_turns=4.0),
                                 dict(fast_turns=float("nan")), dict(original_len=0)])
def test_frequency_ramps_that_are_none(bad):
    with pytest.raises(ValueError):
        api.rope_frequencies(64, scaling="by_parts", factor=4.0, **bad)


@pytest.mark.parametrize("n_seqs,total_q,q_heads,heads,keys", [(16, 512, 16, 2, 32768), (70, 8960, 1, 1, 32768), (3, 300, 4, 4, 9000)])
def test_workspace_of_unlike_sequences(n_seqs, total_q, q_heads, heads, keys):
    # however long one of them may be, there are no more items than queries and sequences make, and
    # no more parts of them than two rounds of SMs or twice the items
    qbuild.build()
    prm = qvg.qvg_page_attention_params(
        n_seqs=n_seqs, n_q_heads=q_heads, n_heads=heads, d=128, page_tokens=64, format=qvg.QVG_PAGE_BF16, q_dtype=qvg.QVG_BF16,
        out_dtype=qvg.QVG_BF16, n_pages=4096, max_pages=keys // 64, causal=1, window=0, total_q=total_q, max_q=total_q, max_kv=keys,
        scale=0.1, q_token_stride=q_heads * 128, q_head_stride=128, o_token_stride=q_heads * 128, o_head_stride=128)
    need = qvg.qvg_page_attention_workspace_bytes(prm)
    items = (total_q * (q_heads // heads) // 256 + n_seqs) * heads
    part = 256 * (128 + 2) * 4
    assert need > 0 and need % part == 0
    assert need // part <= max(8 * 152, 2 * items)
    assert need // part % items == 0
