"""The paged cache, the attention over it and the compression together, as the example runs
them, on a stream small enough to follow in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import pages_model as pm
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("paged_stream", os.path.join(ROOT, "examples", "paged_stream.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["paged_stream"] = m  # (dataclasses look their module up)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_stream_of_chunks(example, fmt):
    s = example.make_stream(heads=2, grid=(2, 6, 8), window=2, chunks=5, fmt=fmt, page=16, C=8)
    freqs, _ = api.rope_frequencies(128, sections=(22, 21, 21))
    read = []  # what each chunk stands for once it is in the pages
    for k in range(5):
        Q, K, V = example.inputs(s, k, "cuda")
        pos = example.positions(s, "cpu")
        out = example.step(s, Q, K, V)
        assert s.packed == max(0, k - 2) and len(s.table) == min(k + 1, 3) * 6
        table = torch.tensor([s.table], dtype=torch.int32)
        n = len(s.table) * 16
        Kp = pm.pool_rows(s.pages.k, s.pages.k_scale, table[0], n, 16)
        Vp = pm.pool_rows(s.pages.v, s.pages.v_scale, table[0], n, 16)
        # the newest chunk's keys are its turned keys, its values its values, to the format's half
        # step: of the value (e4m3 2^-4, bf16 2^-8), of the largest over 127 (int8), of a
        # smallest step (e4m3: 2^-9 / 448 of the largest)
        want, err = pm.rotate(K.cpu(), pos, freqs.tolist(), s.rope.sections, True)
        for got, x, e in ((Kp[:, -96:], want.transpose(0, 1), err.transpose(0, 1)),
                          (Vp[:, -96:], V.double().cpu().transpose(0, 1), 0.0)):
            top = x.abs().amax(-1, keepdim=True)
            half = {"bf16": x.abs() * 2.0 ** -8, "int8": top / 254,
                    "e4m3": torch.maximum(x.abs() * 2.0 ** -4, top * 2.0 ** -10 / 448)}[fmt]
            assert bool(((got - x).abs() <= half * (1 + 2.0 ** -7) + 2 * e + top * 2.0 ** -21).all())
        read.append(torch.stack([Kp[:, -96:], Vp[:, -96:]], 1).flatten(0, 1))
        # every query of the chunk sees all that is cached
        Qr = api.rope(Q, pos.cuda(), s.rope).double().cpu()
        u_p = pm.HALF_EPS[torch.bfloat16 if fmt == "bf16" else torch.float16]
        u_kv = 0.0 if fmt == "bf16" else 2.0 ** -11
        for h in range(2):
            o, _, bound, _ = pm.attend(Qr[:, h], Kp[h], Vp[h], 128 ** -0.5, False, 0, u_p, torch.bfloat16, u_kv, u_kv)
            assert bool(((out[:, h].double().cpu() - o).abs() <= bound).all())
    # the compressed chunks are what the compression gives for the rows that were read back
    c = s.compressed
    alone = api.allocate(4, c.capacity, c.C, c.T, c.bits, c.group, c.n_tables)
    for k in range(2):
        warm = dict(warm=alone.centroids[:, k - 1], warm_stride=alone.centroids.stride(0)) if k else {}
        X = read[k].float().to(torch.bfloat16).cuda()
        api.quantize(X, c.C, c.T, c.bits, c.group, iters=2 if k else 10, seed=1, out=alone,
                     token_offset=k * 96, table_index=k, **warm)
    got = api.dequantize(c, N=192, chunk_len=96, out_dtype=torch.float32)
    want = api.dequantize(alone, N=192, chunk_len=96, out_dtype=torch.float32)
    assert torch.equal(got, want)


def test_a_chunk_must_fill_its_pages(example):
    with pytest.raises(ValueError):
        example.make_stream(heads=1, grid=(1, 3, 5), page=16)
