"""Host-only checks of the paged-cache entry points: struct layouts, refusals before any device
work, the frequency tables, and CPU models of the code conversions."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
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
    buf = (ctypes.c_ubyte * 4096)()
    base = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    yield base
    del buf


STRUCTS = ("qvg_pages", "qvg_rotary", "qvg_rope_params", "qvg_page_write_params",
           "qvg_page_read_params", "qvg_page_attention_params")


def test_struct_layouts(tmp_path):
    lines = []
    for s in STRUCTS:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (s, s))
        for f, _ in getattr(qvg, s)._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (s, f, s, f))
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "qvg.h"\n'
                   'int main(void) {\n%s\nreturn 0;\n}\n' % "\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")], check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, value = line.split()
        cls, _, field = name.partition(".")
        st = getattr(qvg, cls)
        assert int(value) == (getattr(st, field).offset if field else ctypes.sizeof(st)), name


def _rotary(mem, **kw):
    d = dict(rot_dim=64, interleaved=0, n_axes=1, sections=(32, 0, 0, 0), mscale=1.0, pos_stride=0,
             positions=mem, freqs=mem)
    d.update(kw)
    return qvg.qvg_rotary(**d)


BAD_ROTARY = [
    (dict(rot_dim=0), 2), (dict(rot_dim=136), 2), (dict(rot_dim=60, sections=(30, 0, 0, 0)), 2),
    (dict(interleaved=2), 2), (dict(n_axes=0), 2), (dict(n_axes=5), 2),
    (dict(sections=(31, 0, 0, 0)), 1), (dict(n_axes=2, sections=(33, -1, 0, 0), pos_stride=99), 1),
    (dict(n_axes=2, sections=(16, 16, 0, 0), pos_stride=9), 1),
    (dict(mscale=float("nan")), 1), (dict(mscale=float("inf")), 1), (dict(positions=None), 1),
    (dict(freqs=None), 1),
]


def test_rope_refusals(lib, mem, monkeypatch):
    def prm(**kw):
        d = dict(n_tokens=10, n_heads=2, d=128, dtype=qvg.QVG_BF16, backward=0, x_token_stride=256,
                 x_head_stride=128, y_token_stride=256, y_head_stride=128)
        d.update(kw)
        return qvg.qvg_rope_params(**d)
    for bad, code in BAD_ROTARY:
        assert qvg.qvg_rope(prm(), _rotary(mem, **bad), mem, mem, None) == code, bad
    assert qvg.qvg_rope(prm(), _rotary(mem, positions=mem + 4), mem, mem, None) == 1
    assert qvg.qvg_rope(prm(), _rotary(mem, freqs=mem + 8), mem, mem, None) == 1
    for bad, code in ((dict(d=64), 2), (dict(dtype=3), 2), (dict(backward=2), 2), (dict(n_tokens=-1), 1),
                      (dict(n_heads=0), 1), (dict(x_token_stride=-8), 1), (dict(x_head_stride=4), 1),
                      (dict(y_head_stride=0), 1), (dict(y_token_stride=64), 1), (dict(n_tokens=1 << 40), 2)):
        assert qvg.qvg_rope(prm(**bad), _rotary(mem), mem, mem, None) == code, bad
    assert qvg.qvg_rope(prm(), _rotary(mem), None, mem, None) == 1
    assert qvg.qvg_rope(prm(), _rotary(mem), mem, mem + 8, None) == 1
    assert qvg.qvg_rope(None, _rotary(mem), mem, mem, None) == 1
    assert qvg.qvg_rope(prm(), None, mem, mem, None) == 1
    # nothing to do needs no pointers and no device
    assert qvg.qvg_rope(prm(n_tokens=0), _rotary(mem, positions=None, freqs=None), None, None, None) == 0
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")
    assert qvg.qvg_rope(prm(d=64), _rotary(mem), mem, mem, None) == 2
    assert qvg.qvg_rope(prm(), _rotary(mem), mem, mem, None) == qvg.QVG_ERR_CUDA


POOL_BAD = [(dict(d=64), 2), (dict(page_tokens=8), 2), (dict(page_tokens=48), 2),
            (dict(page_tokens=256), 2), (dict(format=4), 2), (dict(format=-1), 2), (dict(n_pages=0), 1),
            (dict(n_heads=0), 1), (dict(n_heads=40000), 2), (dict(n_pages=1 << 27), 2)]


def test_page_write_refusals(lib, mem, monkeypatch):
    def prm(**kw):
        d = dict(n_tokens=10, n_heads=2, d=128, page_tokens=16, format=qvg.QVG_PAGE_E4M3, n_pages=4,
                 in_dtype=qvg.QVG_BF16, k_token_stride=256, k_head_stride=128, v_token_stride=256,
                 v_head_stride=128)
        d.update(kw)
        return qvg.qvg_page_write_params(**d)
    good = qvg.qvg_pages(mem, mem, mem, mem)

    def call(p=None, K=mem, V=mem, slots=mem, rot=None, pages=good):
        return qvg.qvg_page_write(prm() if p is None else p, K, V, slots, rot, pages, None, None)
    for bad, code in POOL_BAD + [(dict(in_dtype=3), 2), (dict(n_tokens=-1), 1), (dict(k_token_stride=4), 1),
                                 (dict(v_head_stride=-128), 1)]:
        assert call(prm(**bad)) == code, bad
    for bad, code in BAD_ROTARY:
        assert call(rot=_rotary(mem, **bad)) == code, bad
    for pages in (qvg.qvg_pages(None, mem, mem, mem), qvg.qvg_pages(mem, mem + 8, mem, mem),
                  qvg.qvg_pages(mem, mem, None, mem), qvg.qvg_pages(mem, mem, mem, None), None):
        assert call(pages=pages) == 1
    assert call(K=None) == 1 and call(V=mem + 2) == 1 and call(slots=None) == 1 and call(slots=mem + 4) == 1
    assert qvg.qvg_page_write(None, mem, mem, mem, None, good, None, None) == 1
    assert call(prm(n_tokens=0), K=None, V=None, slots=None) == 0
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")
    assert call() == qvg.QVG_ERR_CUDA
    assert call(prm(format=qvg.QVG_PAGE_F16), pages=qvg.qvg_pages(mem, mem, None, None)) == qvg.QVG_ERR_CUDA


def test_page_read_refusals(lib, mem, monkeypatch):
    def prm(**kw):
        d = dict(n_seqs=2, n_heads=2, d=128, page_tokens=16, format=qvg.QVG_PAGE_E4M3,
                 out_dtype=qvg.QVG_BF16, n_pages=4, max_pages=3, first=0, count=20,
                 x_seq_stride=4 * 20 * 128, x_tensor_stride=20 * 128)
        d.update(kw)
        return qvg.qvg_page_read_params(**d)
    good = qvg.qvg_pages(mem, mem, mem, mem)

    def call(p=None, table=mem, lens=mem, X=mem, pages=good):
        return qvg.qvg_page_read(prm() if p is None else p, pages, table, lens, X, None, None)
    for bad, code in POOL_BAD + [(dict(out_dtype=5), 2), (dict(n_seqs=0), 1), (dict(n_seqs=70000), 2),
                                 (dict(max_pages=0), 1), (dict(first=-1), 1), (dict(count=-1), 1),
                                 (dict(first=1 << 31), 2), (dict(x_tensor_stride=20 * 128 - 8), 1),
                                 (dict(x_seq_stride=0), 1), (dict(x_tensor_stride=20 * 128 + 4), 1)]:
        assert call(prm(**bad)) == code, bad
    assert call(table=None) == 1 and call(lens=None) == 1 and call(X=None) == 1 and call(X=mem + 8) == 1
    assert call(pages=qvg.qvg_pages(mem, mem, None, mem)) == 1
    assert qvg.qvg_page_read(None, good, mem, mem, mem, None, None) == 1
    assert call(prm(count=0), table=None, lens=None, X=None) == 0
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")
    assert call() == qvg.QVG_ERR_CUDA


def _attention(**kw):
    d = dict(n_seqs=2, n_q_heads=4, n_heads=2, d=128, page_tokens=16, format=qvg.QVG_PAGE_E4M3,
             q_dtype=qvg.QVG_BF16, out_dtype=qvg.QVG_BF16, n_pages=40, max_pages=20, causal=1, window=0,
             total_q=6, max_q=3, max_kv=300, scale=0.1, q_token_stride=512, q_head_stride=128,
             o_token_stride=512, o_head_stride=128)
    d.update(kw)
    return qvg.qvg_page_attention_params(**d)


ATTENTION_BAD = POOL_BAD + [
    (dict(n_seqs=0), 1), (dict(n_seqs=70000), 2), (dict(n_q_heads=0), 1), (dict(n_q_heads=5), 1),
    (dict(n_q_heads=2 * 129), 2), (dict(q_dtype=qvg.QVG_F32), 2), (dict(out_dtype=3), 2),
    (dict(format=qvg.QVG_PAGE_F16), 2), (dict(format=qvg.QVG_PAGE_BF16, q_dtype=qvg.QVG_F16), 2),
    (dict(max_pages=0), 1), (dict(causal=2), 2), (dict(window=-1), 1), (dict(total_q=-1), 1),
    (dict(max_q=0), 1), (dict(max_kv=-1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q_token_stride=-512), 1), (dict(q_head_stride=4), 1),
    (dict(o_head_stride=0), 1), (dict(o_token_stride=64), 1), (dict(total_q=1 << 40), 2),
    (dict(max_q=1 << 30), 2)]


def test_page_attention_refusals(lib, mem, monkeypatch):
    good = qvg.qvg_pages(mem, mem, mem, mem)

    def call(p=None, Q=mem, pages=good, table=mem, lens=mem, cu=mem, O=mem, lse=None, ws=mem, n=1 << 40):
        return qvg.qvg_page_attention(_attention() if p is None else p, Q, pages, table, lens, cu, O, lse,
                                      ws, n, None, None)
    for bad, code in ATTENTION_BAD:
        assert call(_attention(**bad)) == code, bad
        assert qvg.qvg_page_attention_workspace_bytes(_attention(**bad)) == 0, bad
    assert call(Q=None) == call(Q=mem + 2) == call(O=None) == call(O=mem + 8) == 1
    assert call(table=None) == call(lens=None) == call(lse=mem + 2) == call(pages=None) == 1
    assert call(pages=qvg.qvg_pages(mem, mem, mem, None)) == 1
    assert call(_attention(total_q=5), cu=None) == 1  # unequal shares need cu_q
    assert qvg.qvg_page_attention(None, mem, good, mem, mem, mem, mem, None, mem, 1, None, None) == 1
    assert qvg.qvg_page_attention_workspace_bytes(None) == 0
    # long keys and few rows: the keys are split many ways, which needs workspace
    long = _attention(n_seqs=1, total_q=3, n_pages=2000, max_pages=1250, max_kv=20000)
    need = qvg.qvg_page_attention_workspace_bytes(long)
    rows = 2 * 16  # a 16-row tile of either key/value head, for each split
    assert need > 0 and need % (rows * (128 + 2) * 4) == 0
    assert call(long, n=need - 1) == call(long, ws=None) == call(long, ws=mem + 4) == qvg.QVG_ERR_WORKSPACE
    assert call(_attention(total_q=0, max_q=0), Q=None, table=None, lens=None, O=None, ws=None, n=0) == 0
    monkeypatch.setenv("QVG_FAULT_INJECT", "launch")
    assert call(long, n=need) == qvg.QVG_ERR_CUDA
    assert call(long, n=need - 1) == qvg.QVG_ERR_WORKSPACE


def test_rope_frequencies():
    f, m = api.rope_frequencies(64, base=5e5)
    assert m == 1.0 and f[0] == 1.0 and math.isclose(f[31], 5e5 ** (-31 / 32))
    f3, _ = api.rope_frequencies(128, sections=(22, 21, 21))
    assert f3[22] == 1.0 and f3[43] == 1.0 and math.isclose(f3[23], 1e4 ** (-1 / 21))
    lin, _ = api.rope_frequencies(64, base=5e5, scaling="linear", factor=4)
    assert torch.allclose(lin * 4, f, rtol=1e-15)
    st, _ = api.rope_frequencies(64, scaling="stretched", factor=4)
    base, _ = api.rope_frequencies(64)
    assert st[0] == 1.0 and math.isclose(st[31] * 4, base[31])
    yarn, ym = api.rope_frequencies(64, scaling="by_parts", factor=4)
    turns = 4096 * base / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], base[turns > 32])
    assert torch.allclose(yarn[turns < 1] * 4, base[turns < 1], rtol=1e-15)
    assert math.isclose(ym, 0.1 * math.log(4) + 1)
    for bad in (dict(scaling="cubic"), dict(factor=0.5), dict(base=-1.0), dict(sections=(1, 2))):
        with pytest.raises(ValueError):
            api.rope_frequencies(64, **bad)
    with pytest.raises(ValueError):
        api.rope_table(64, freqs=f, base=2.0, device="cpu")
    with pytest.raises(ValueError):
        api.rope_table(64, freqs=[1.0] * 31, device="cpu")
    with pytest.raises(ValueError):
        api.rope_table(4, freqs=[1.0, float("nan")], device="cpu")


@pytest.mark.parametrize("pos", [0, 1, -1, 123456789, -(2 ** 31), 2 ** 40 + 7])
def test_wrapped_angles(pos):
    """position * frequency mod 2^64, its top word a signed fraction of a turn: the angle, to
    2^-32 of a turn and what the frequency's own rounding gives."""
    for f in (1.0, 0.1234567, 1e4 ** (-13 / 64), 7.5):
        turns = f / (2 * math.pi)  # rounded to double here as in the table
        word = round(Fraction(turns) * 2 ** 64) % 2 ** 64
        w = word * (pos % 2 ** 64) % 2 ** 64
        top = w >> 32
        frac = (top - 2 ** 32 if top >= 2 ** 31 else top) / 2 ** 32
        want = Fraction(turns) * pos
        off = abs((want - Fraction(frac)) - round(want - Fraction(frac)))
        assert off <= 2 ** -32 + abs(pos) * 2.0 ** -65


def _bf16(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def test_code_conversions_are_exact():
    """The bit steps that widen 8-bit codes, on all 256 of them."""
    b = np.arange(256, dtype=np.uint32)
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    t = b << 8
    fields = (t & 0x8000) | ((t >> 4) & 0x07F0)
    got = _bf16(fields).astype(np.float64) * 2.0 ** 120
    ok = (b & 0x7F) != 0x7F  # the NaN codes are never stored
    assert np.array_equal(got[ok], want[ok].astype(np.float64))
    assert float(_bf16(0x7B80)) == 2.0 ** 120
    signed = b.astype(np.uint8).view(np.int8).astype(np.float64)
    t = 0x4300 | b
    assert np.array_equal(_bf16(t & 0xFF7F).astype(np.float64) - _bf16(t & 0xFF80), signed)
    half = (0x6400 | (b ^ 0x80)).astype(np.uint16).view(np.float16).astype(np.float64)
    assert np.array_equal(half - 1152.0, signed)


def test_handles_refuse_wrong_shapes():
    with pytest.raises(ValueError):
        api.PagedKV(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))
    with pytest.raises(ValueError):  # on the CPU
        api.PagedKV(torch.zeros(2, 1, 16, 128).half(), torch.zeros(2, 1, 16, 128).half())
    with pytest.raises(ValueError):
        api.allocate_pages(2, 1, 16, torch.float32, device="cpu")
    with pytest.raises(ValueError):
        api.rope(torch.zeros(2, 1, 128), torch.zeros(2, dtype=torch.int64), None)
