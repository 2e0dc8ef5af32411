"""Host-only checks of 4-bit pages: the definition's model, and refusals before any device work."""
import ctypes

import pytest
import torch

from tests import pages4_model as m4
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qvg.load()


@pytest.fixture()
def mem():
    buf = (ctypes.c_ubyte * 4096)()
    yield ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    del buf


@pytest.mark.parametrize("fmt", [m4.E2M1, m4.INT4])
def test_the_model_rounds_to_the_nearest_code_and_halves_to_the_even_one(fmt):
    top = m4.TOP[fmt]
    codes = [c for c in range(16) if not (fmt is m4.INT4 and c == 8) and not (fmt is m4.E2M1 and c == 8)]
    x = torch.zeros(128)
    x[:len(codes)] = torch.tensor([m4.VALUES[fmt][c] for c in codes])
    x[16:32] = x[:16] / 2
    raw, t, s = m4.stored(x, fmt)
    assert float(s) == torch.tensor(top / (64 * top)).float() and t.float().tolist() == [64.0, 32.0] + [0.0] * 6
    assert torch.equal(m4.decoded(raw, t, s, fmt), x.double())
    # between neighbours: 2.5 of E2M1 goes to 2, 3.5 to 4, 5 to 4; 2.5 of INT4 to 2, 3.5 to 4
    x = torch.zeros(128)
    half = {m4.E2M1: ([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], [6, 0, 1, 1, 2, 2, 4, 4]),
            m4.INT4: ([7, 0.5, 1.5, 2.5, 3.5, 4.5, 5.5, 6.5], [7, 0, 2, 2, 4, 4, 6, 6])}[fmt]
    x[:8], x[16:24] = torch.tensor(half[0]), -torch.tensor(half[0])
    y = m4.decoded(*m4.stored(x, fmt), fmt)
    assert y[:8].tolist() == half[1] and (-y[16:24]).tolist() == half[1]


@pytest.mark.parametrize("fmt", [m4.E2M1, m4.INT4])
def test_the_models_error_is_what_the_format_allows(fmt):
    # half a step of a code at the group's scale; what is cut at the largest code, up to a
    # sixteenth of it, is no more than that
    x = torch.randn((200, 128), generator=torch.Generator().manual_seed(1))
    raw, t, s = m4.stored(x, fmt)
    y = m4.decoded(raw, t, s, fmt)
    unit = (t.double() * s.double()[:, None]).repeat_interleave(16, -1)
    step = torch.where(x.abs() / unit < 2, 0.5, torch.where(x.abs() / unit < 4, 1.0, 2.0)) if fmt is m4.E2M1 else 1.0
    assert bool(((y - x).abs() <= unit * (step / 2 + 2.0 ** -20)).all())


def test_write_read_and_attention_refuse_what_4_bit_pages_lack(lib, mem, monkeypatch):
    w = dict(n_tokens=10, n_heads=2, d=128, page_tokens=16, n_pages=4, in_dtype=qvg.QVG_BF16, k_token_stride=256,
             k_head_stride=128, v_token_stride=256, v_head_stride=128)
    r = dict(n_seqs=2, n_heads=2, d=128, page_tokens=16, out_dtype=qvg.QVG_BF16, n_pages=4, max_pages=3, first=0, count=20,
             x_seq_stride=4 * 20 * 128, x_tensor_stride=20 * 128)
    a = dict(n_seqs=2, n_q_heads=4, n_heads=2, d=128, page_tokens=16, q_dtype=qvg.QVG_BF16, out_dtype=qvg.QVG_BF16,
             n_pages=4, max_pages=3, causal=1, window=0, total_q=2, max_q=1, max_kv=40, scale=0.1, q_token_stride=512,
             q_head_stride=128, o_token_stride=512, o_head_stride=128)

    def codes(fmt, pages):
        return (qvg.qvg_page_write(qvg.qvg_page_write_params(format=fmt, **w), mem, mem, mem, None, pages, None, None),
                qvg.qvg_page_read(qvg.qvg_page_read_params(format=fmt, **r), pages, mem, mem, mem, None, None),
                qvg.qvg_page_attention(qvg.qvg_page_attention_params(format=fmt, **a), mem, pages, mem, mem, None, mem, None,
                                       mem, 4096, None, None))
    good = qvg.qvg_pages(mem, mem, mem, mem, mem, mem)
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")  # what is accepted ends there, before the device
    for fmt in (qvg.QVG_PAGE_E2M1, qvg.QVG_PAGE_INT4):
        assert codes(fmt, good) == (qvg.QVG_ERR_CUDA,) * 3
        for bad in (qvg.qvg_pages(mem, mem, mem, mem), qvg.qvg_pages(mem, mem, mem, mem, mem, None),
                    qvg.qvg_pages(mem, mem, mem, mem, None, mem), qvg.qvg_pages(mem, mem, mem, mem, mem + 8, mem),
                    qvg.qvg_pages(mem, mem, None, mem, mem, mem), qvg.qvg_pages(mem, mem, mem, mem + 4, mem, mem)):
            assert codes(fmt, bad) == (1, 1, 1)
    for fmt in (4, 5, 6, 7, 10, 11):
        assert codes(fmt, good) == (2, 2, 2)
    # the other formats read no group scales
    assert codes(qvg.QVG_PAGE_INT8, qvg.qvg_pages(mem, mem, mem, mem, mem + 1, None)) == (qvg.QVG_ERR_CUDA,) * 3


def test_pages_that_do_not_fit_together():
    # (host tensors: refused for their shapes and types before their place)
    def pages(dtype=m4.E2M1, width=64, group=8, gtype=torch.float8_e4m3fn):
        k = torch.zeros((2, 1, 16, width), dtype=torch.uint8).view(dtype)
        s = torch.zeros((2, 1, 16))
        t = torch.zeros((2, 1, 16, group), dtype=torch.uint8).view(gtype)
        return api.PagedKV(k, k, s, s, t, t)
    for bad in (dict(width=128), dict(dtype=m4.INT4, width=32), dict(group=4), dict(gtype=torch.uint8), dict(dtype=torch.int8)):
        with pytest.raises(ValueError):
            pages(**bad)
