"""What the paged-cache calls refuse without a GPU in the machine."""
import pytest
import torch

from video_kv_cache_gb300 import api


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
