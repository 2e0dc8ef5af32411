"""Host-only checks of the calls on the pages of sequences: the struct's layout, and refusals before any
device work."""
import ctypes
import os
import subprocess

import pytest
import torch

from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qvg.load()


@pytest.fixture()
def mem():
    buf = (ctypes.c_ubyte * 8192)()
    yield ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    del buf


def test_struct_layout(tmp_path):
    fields = [f for f, _ in qvg.qvg_page_table_params._fields_]
    lines = ['printf("%zu\\n", sizeof(qvg_page_table_params));']
    lines += ['printf("%%zu\\n", offsetof(qvg_page_table_params, %s));' % f for f in fields]
    (tmp_path / "l.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "qvg.h"\n'
                                  'int main(void) {\n%s\nreturn 0;\n}\n' % "\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(qvg.qvg_page_table_params)] + \
        [getattr(qvg.qvg_page_table_params, f).offset for f in fields]


def _prm(**kw):
    return qvg.qvg_page_table_params(**dict(dict(n_seqs=4, n_heads=2, d=128, page_tokens=16, format=qvg.QVG_PAGE_INT8, max_pages=5,
                                                 n_pages=9, total=10, out_pages=3), **kw))


def test_refusals(lib, mem, monkeypatch):
    pages, other = qvg.qvg_pages(mem, mem, mem, mem), qvg.qvg_pages(*(mem + (k << 20) for k in (1, 2, 3, 4)))  # (never read)
    far = mem + 4096

    def append(p=None, g=pages, refs=mem, table=mem, lens=mem, counts=mem, slots=mem, pos=mem, copies=mem, ws=mem, size=4096):
        return qvg.qvg_page_append(_prm() if p is None else p, g, refs, table, lens, counts, slots, pos, copies, ws, size, None, None)

    def fork(p=None, g=pages, refs=mem, table=mem, lens=mem, parents=mem, copies=mem, ws=mem, size=4096):
        return qvg.qvg_page_fork(_prm() if p is None else p, g, refs, table, lens, parents, copies, ws, size, None, None)

    def free(p=None, refs=mem, table=mem, lens=mem, first=mem, last=None):
        return qvg.qvg_page_free(_prm() if p is None else p, refs, table, lens, first, last, None, None)

    def compact(p=None, g=pages, refs=mem, table=mem, lens=mem, to=other, out_table=far, out_refs=far, live=mem, ws=mem, size=4096):
        return qvg.qvg_page_compact(_prm() if p is None else p, g, refs, table, lens, to, out_table, out_refs, live, ws, size, None, None)

    def copies(p=None, n=3, g=pages, src=mem, dst=mem, rows=None, to=pages, to_pages=9):
        return qvg.qvg_page_copy(_prm() if p is None else p, n, g, src, dst, rows, to, to_pages, None, None)
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")  # what is accepted ends there, before the device
    for call in (append, fork, free, compact, copies):
        assert call() == qvg.QVG_ERR_CUDA
        for bad, code in ((dict(d=64), 2), (dict(page_tokens=24), 2), (dict(format=4), 2), (dict(n_pages=0), 1), (dict(n_heads=0), 1),
                          (dict(n_pages=1 << 27), 2)):
            assert call(_prm(**bad)) == code, bad
    for call in (append, fork, free, compact):
        for bad, code in ((dict(n_seqs=0), 1), (dict(n_seqs=65536), 2), (dict(max_pages=0), 1), (dict(max_pages=(1 << 23) + 1), 2),
                          (dict(total=-1), 1), (dict(total=1 << 31), 2), (dict(out_pages=-1), 1), (dict(out_pages=1 << 30), 2)):
            assert call(_prm(**bad)) == code, bad
        for bad in (dict(refs=None), dict(refs=mem + 4), dict(table=None), dict(table=mem + 2), dict(lens=None)):
            assert call(**bad) == 1, bad
    for call, p in ((append, dict(n_seqs=1025, out_pages=0)), (fork, dict(n_seqs=1025, out_pages=0)), (compact, {})):
        assert call(g=qvg.qvg_pages(mem, None, mem, mem)) == 1
        need = qvg.qvg_page_table_workspace_bytes(_prm(**p))
        assert need > 0 and call(_prm(**p), size=need) == qvg.QVG_ERR_CUDA
        for bad in (dict(ws=None), dict(ws=mem + 8), dict(size=need - 1)):
            assert call(_prm(**p), **dict(dict(size=need), **bad)) == qvg.QVG_ERR_WORKSPACE
    for call in (append, fork):  # the wants of few sequences take none
        assert qvg.qvg_page_table_workspace_bytes(_prm(out_pages=0)) == 0 and call(ws=None, size=0) == qvg.QVG_ERR_CUDA
    assert append(counts=None) == append(slots=None) == append(pos=mem + 4) == append(copies=mem + 2) == 1
    assert append(copies=None) == qvg.QVG_ERR_CUDA and fork(copies=None) == 1
    assert append(_prm(total=0), slots=None, pos=None) == qvg.QVG_ERR_CUDA
    assert fork(parents=None) == fork(copies=mem + 1) == 1
    assert free(first=None) == free(first=mem + 2) == free(last=mem + 2) == 1 and free(first=None, last=mem) == qvg.QVG_ERR_CUDA
    assert compact(_prm(out_pages=0)) == compact(to=pages) == compact(out_table=mem) == compact(out_refs=mem) == compact(live=None) == 1
    inside = qvg.qvg_pages(mem + 8 * 2 * 16 * 128, mem + (2 << 20), mem + (3 << 20), mem + (4 << 20))  # its last page of keys
    behind = qvg.qvg_pages(mem + 9 * 2 * 16 * 128, mem + (2 << 20), mem + (3 << 20), mem + (4 << 20))
    assert compact(to=inside) == 1 and compact(to=behind) == qvg.QVG_ERR_CUDA
    assert copies(n=-1) == copies(src=None) == copies(dst=mem + 2) == copies(rows=mem + 1) == copies(to=None) == 1
    assert copies(to_pages=0) == 1 and copies(to_pages=1 << 28) == 2 and copies(n=1 << 31) == 2
    assert copies(n=0, src=None, dst=None) == 0
    monkeypatch.delenv("QVG_FAULT_INJECT")
    assert qvg.qvg_page_table_workspace_bytes(_prm()) >= 9 * 4 + 3 * 4
    assert qvg.qvg_page_table_workspace_bytes(_prm(d=1)) == 0


def test_host_tensors_are_refused():
    kv = type("Pages", (), dict(k=torch.zeros(1), heads=2, gpu=-1, n_pages=3))()
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: api.page_append(kv, i, i, i, i, 0), lambda: api.page_fork(kv, i, i, i, i),
                 lambda: api.page_free(kv, i, i, i, first=i), lambda: api.page_copy(kv, i, i), lambda: api.page_compact(kv, i, i, i, kv)):
        with pytest.raises(ValueError):
            call()
