"""What the paged-cache calls refuse before anything is launched, on a GPU machine: tensors in other
places than the call's, of the wrong type or shape."""
import copy
import pickle

import pytest
import torch

from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


@pytest.fixture()
def made():
    n, heads = 20, 2
    kv = api.allocate_pages(4, heads, 16, BF)
    kv.k.zero_()
    kv.v.zero_()
    x = torch.zeros((n, heads, 128), dtype=BF, device="cuda")
    return dict(kv=kv, x=x, pos=torch.arange(n).cuda(), slots=torch.arange(n).cuda(), rope=api.rope_table(64),
                table=torch.tensor([[0, 1, 2]], dtype=torch.int32).cuda(), lens=torch.tensor([n], dtype=torch.int32).cuda(),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _attend(m, **kw):
    a = dict(Q=m["x"], kv=m["kv"], page_table=m["table"], seq_lens=m["lens"], status=m["status"])
    a.update(kw)
    return api.page_attention(**a)


def _write(m, **kw):
    a = dict(kv=m["kv"], K=m["x"], V=m["x"], slots=m["slots"], rope=m["rope"], positions=m["pos"], status=m["status"])
    a.update(kw)
    return api.page_write(**a)


def _read(m, **kw):
    a = dict(kv=m["kv"], page_table=m["table"], seq_lens=m["lens"], count=20, status=m["status"])
    a.update(kw)
    return api.page_read(**a)


def _rope(m, **kw):
    a = dict(X=m["x"], positions=m["pos"], table=m["rope"])
    a.update(kw)
    return api.rope(**a)


def test_tensors_off_the_gpu_are_refused(made):
    m = made
    for call in (_attend, _write, _read, _rope):
        call(m)
    host = m["x"].cpu()
    word = torch.zeros(1, dtype=torch.int32)
    for bad in (dict(Q=host), dict(page_table=m["table"].cpu()), dict(seq_lens=m["lens"].cpu()), dict(status=word),
                dict(status=word.cuda().float()), dict(status=word.cuda()[:0]), dict(out=host),
                dict(lse=torch.zeros((20, 2))), dict(cu_q=torch.tensor([0, 20], dtype=torch.int32)),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                dict(workspace=torch.empty((1 << 12, 2), dtype=torch.uint8, device="cuda")[:, 0])):
        with pytest.raises(ValueError):
            _attend(m, **bad)
    for bad in (dict(K=host), dict(V=host), dict(slots=m["slots"].cpu()), dict(positions=m["pos"].cpu()), dict(status=word)):
        with pytest.raises(ValueError):
            _write(m, **bad)
    for bad in (dict(page_table=m["table"].cpu()), dict(seq_lens=m["lens"].cpu()), dict(status=word),
                dict(out=torch.zeros((1, 4, 20, 128)))):
        with pytest.raises(ValueError):
            _read(m, **bad)
    for bad in (dict(X=host), dict(positions=m["pos"].cpu()), dict(out=host)):
        with pytest.raises(ValueError):
            _rope(m, **bad)
    torch.cuda.synchronize()
    assert int(m["status"]) == 0


def test_tensors_of_another_gpu_are_refused(made, monkeypatch):
    # with one GPU in hand: the tensors' GPU is not the current one
    m = made
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (_attend, _write, _read, _rope):
        with pytest.raises(ValueError):
            call(m)


def test_no_sequences_are_refused(made):
    m = made
    none, no_pages = torch.zeros((0, 3), dtype=torch.int32, device="cuda"), torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    for call in (_attend, _read):
        with pytest.raises(ValueError):
            call(m, page_table=none, seq_lens=m["lens"][:0])
        with pytest.raises(ValueError):
            call(m, page_table=no_pages)
    assert _attend(m, Q=m["x"][:0]).shape == (0, 2, 128)  # no queries are nothing to do


def test_rope_does_not_lose_a_gradient(made):
    m = made
    x = torch.randn((20, 2, 128), device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        api.rope(x, m["pos"], m["rope"])
    with torch.no_grad():
        want = api.rope(x, m["pos"], m["rope"])

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return api.rope(x, m["pos"], m["rope"])

        @staticmethod
        def backward(ctx, dy):
            return api.rope(dy, m["pos"], m["rope"], backward=True)
    y = Turn.apply(x)
    assert torch.equal(y, want)
    dy = torch.randn_like(want)
    y.backward(dy)
    assert torch.equal(x.grad, api.rope(dy, m["pos"], m["rope"], backward=True))


@pytest.mark.parametrize("fmt", [BF, torch.int8])
def test_handles_can_be_copied(made, fmt):
    # a copy is of the pages and the table, not of where they lie
    m = made
    kv = api.allocate_pages(4, 2, 16, fmt)
    x = torch.randn((20, 2, 128), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    api.page_write(kv, x, x, m["slots"], rope=m["rope"], positions=m["pos"])
    want = api.page_attention(x, kv, m["table"], m["lens"])
    for again in (copy.copy(kv), copy.deepcopy(kv), pickle.loads(pickle.dumps(kv))):
        assert torch.equal(api.page_attention(x, again, m["table"], m["lens"]), want)
    far = copy.deepcopy(kv)
    kv.k.zero_()
    assert torch.equal(api.page_attention(x, far, m["table"], m["lens"]), want)
    for rope in (copy.copy(m["rope"]), copy.deepcopy(m["rope"]), pickle.loads(pickle.dumps(m["rope"]))):
        assert torch.equal(api.rope(x, m["pos"], rope), api.rope(x, m["pos"], m["rope"]))
