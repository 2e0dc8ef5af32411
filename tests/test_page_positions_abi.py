"""Host-only check of the positions of sequences' first tokens: an address that cannot hold them is refused
before any device work."""
import ctypes

from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg


def test_starts_are_aligned(monkeypatch):
    qbuild.build()
    qvg.load()
    buf = (ctypes.c_ubyte * 4096)()
    mem = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    pages = qvg.qvg_pages(mem, mem, mem, mem)
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")  # what is accepted ends there, before the device
    for starts, code in ((None, qvg.QVG_ERR_CUDA), (mem + 8, qvg.QVG_ERR_CUDA), (mem + 4, 1)):
        p = qvg.qvg_page_table_params(n_seqs=4, n_heads=2, d=128, page_tokens=16, format=qvg.QVG_PAGE_INT8, max_pages=5,
                                      n_pages=9, total=10, starts=starts)
        assert qvg.qvg_page_append(p, pages, mem, mem, mem, mem, mem, mem, None, None, 0, None, None) == code
        assert qvg.qvg_page_fork(p, pages, mem, mem, mem, mem, mem, None, 0, None, None) == code
        assert qvg.qvg_page_free(p, mem, mem, mem, mem, None, None, None) == code
