"""Host-only check that pages are not packed into memory that they are read from: any array of the one pool
against any of the other, and the tables."""
import ctypes

import pytest

from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

PAGES, OUT, HEADS, PAGE, SEQS, ENTRIES = 9, 3, 2, 16, 4, 5
ROW = {"k": 64, "v": 64, "k_scale": 4, "v_scale": 4, "k_group": 8, "v_group": 8}  # bytes in 4 bits
NAMES = list(ROW)


@pytest.fixture()
def compact(monkeypatch):
    qbuild.build()
    qvg.load()
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")  # what is accepted ends there, before the device
    buf = (ctypes.c_ubyte * 65536)()
    mem = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256

    def call(out=None, table=None, refs=None):
        # (the pools' addresses are compared, never read)
        src = {n: mem + (k + 1 << 24) for k, n in enumerate(NAMES)}
        dst = {n: mem + (k + 33 << 24) for k, n in enumerate(NAMES)}
        out_table, out_refs = mem + 8192, mem + 12288
        if out:
            to, of, off = out
            dst[to] = src[of] + off
        out_table = mem + table if table is not None else out_table
        out_refs = mem + 4096 + refs if refs is not None else out_refs
        p = qvg.qvg_page_table_params(n_seqs=SEQS, n_heads=HEADS, d=128, page_tokens=PAGE, format=qvg.QVG_PAGE_INT4,
                                      max_pages=ENTRIES, n_pages=PAGES, out_pages=OUT)
        return qvg.qvg_page_compact(p, qvg.qvg_pages(*(src[n] for n in NAMES)), mem + 4096, mem, mem + 16384,
                                    qvg.qvg_pages(*(dst[n] for n in NAMES)), out_table, out_refs, mem + 20480, mem + 24576, 4096,
                                    None, None)
    yield call
    del buf


@pytest.mark.parametrize("to", NAMES)
@pytest.mark.parametrize("of", NAMES)
def test_no_array_is_packed_into_one_that_is_read(compact, to, of):
    rows = HEADS * PAGE
    held, taken = ROW[of] * rows * PAGES, ROW[to] * rows * OUT
    assert compact() == qvg.QVG_ERR_CUDA
    for off, code in ((0, 1), (held - 16, 1), (16 - taken, 1), (held, qvg.QVG_ERR_CUDA), (-taken, qvg.QVG_ERR_CUDA)):
        assert compact(out=(to, of, off)) == code, off


def test_no_table_is_written_into_one_that_is_read(compact):
    for off, code in ((0, 1), (4 * SEQS * ENTRIES - 4, 1), (4 * SEQS * ENTRIES, qvg.QVG_ERR_CUDA)):
        assert compact(table=off) == code
    for off, code in ((0, 1), (4 * PAGES - 4, 1), (4 - 4 * OUT, 1), (4 * PAGES, qvg.QVG_ERR_CUDA), (-4 * OUT, qvg.QVG_ERR_CUDA)):
        assert compact(refs=off) == code
