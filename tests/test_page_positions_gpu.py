"""GPU checks of positions in sequences that drop their oldest tokens: they count on, so that new tokens are
turned relative to those that are kept."""
import random

import pytest
import torch

from tests import pages4_model as m4
from tests import test_page_book_gpu as tb
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu
BF, E4, I8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8
ALL = tb.ALL


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


class Model(tb.Model):
    """With the position of each sequence's first token."""

    def __init__(self, kv, rows, entries):
        super().__init__(kv, rows, entries)
        self.start = [0] * rows

    def append(self, counts, total):
        slots, pos, copies, status = super().append(counts, total)
        row = [b for b, c in enumerate(counts) for _ in range(max(0, c))]
        return slots, [p + self.start[row[i]] if p >= 0 else p for i, p in enumerate(pos)], copies, status

    def fork(self, parents):
        was = list(self.size)
        out = super().fork(parents)
        for b, p in enumerate(parents):
            if was[b] == 0 and self.size[b] > 0:
                self.start[b] = self.start[p]
        return out

    def give(self, first, last):
        was = list(self.size)
        super().give(first, last)
        for b, n in enumerate(was):
            if last[b] > 0 and last[b] >= n:
                self.start[b] = 0
            elif first[b] > 0 or last[b] > 0:
                self.start[b] += n - min(max(last[b], 0), n) - self.size[b]


def _append(kv, s, counts, starts):
    status, copies = tb._int([0]), torch.empty((3, len(counts)), dtype=torch.int32, device="cuda")
    slots, pos = api.page_append(kv, *s, tb._int(counts), sum(counts), starts=starts, copies=copies, status=status)
    return slots.tolist(), pos.tolist(), copies.tolist(), int(status)


@pytest.mark.parametrize("pages,rows,entries,most", [
    (60, 7, 12, 16),         # a thread for each sequence
    (90, 7, 20, 60),         # a thread for each token
    (40000, 5, 400, 3000),   # a cluster of CTAs
    (3000, 1100, 6, 30),     # more sequences than shared memory has room for
])
def test_positions_count_on(pages, rows, entries, most):
    r = random.Random(pages)
    page = 16
    kv = tb._filled(pages, 1, page, I8, rows)
    s, m = tb._state(kv, rows, entries), Model(kv, rows, entries)
    starts = torch.zeros(rows, dtype=torch.int64, device="cuda")
    starts[0], m.start[0] = 2 ** 40, 2 ** 40   # a caller's own, past 32 bits
    for step in range(24):
        kind = ("append", "free", "fork")[step % 3]
        if kind == "append":
            counts = [r.choice([0, 1, r.randint(0, most)]) for _ in range(rows)]
            assert _append(kv, s, counts, starts) == m.append(counts, sum(counts)), step
        elif kind == "fork":
            old = [b for b in range(rows) if m.size[b]]
            parents = [r.choice(old) if old and not m.size[b] and r.random() < 0.7 else -1 for b in range(rows)]
            status = tb._int([0])
            api.page_fork(kv, *s, tb._int(parents), starts=starts, status=status)
            assert int(status) == m.fork(parents)[1], step
        else:
            first = [r.choice([0, 0, r.randint(0, 3 * page), most, ALL]) for _ in range(rows)]
            last = [r.choice([0, 0, 0, 1, r.randint(0, page), ALL]) for _ in range(rows)]
            which = r.choice(["both", "first", "last"])
            api.page_free(kv, *s, first=tb._int(first) if which != "last" else None,
                          last=tb._int(last) if which != "first" else None, starts=starts)
            m.give(first if which != "last" else [0] * rows, last if which != "first" else [0] * rows)
        assert starts.tolist() == m.start, (step, kind)
    m.check(kv, *s)
    assert max(m.start[1:]) > 0


@pytest.mark.parametrize("fmt", [BF, E4, m4.E2M1, m4.INT4])
@pytest.mark.parametrize("chunk,window", [(1, 20), (48, 96), (37, 100)])
def test_a_sliding_window_attends_as_over_a_cache_of_its_own(fmt, chunk, window):
    # chunks are turned, written and attended to, the oldest pages dropped before each; every step against a
    # fresh cache that holds the kept tokens at their positions
    heads, page, steps = 2, 16, 12 if chunk > 1 else 70
    g = torch.Generator().manual_seed(chunk)
    kv = api.allocate_pages(24, heads, page, fmt)
    s, starts = tb._state(kv, 1, 12), torch.zeros(1, dtype=torch.int64, device="cuda")
    rope = api.rope_table(128, base=100.0)
    x = torch.randn((chunk * steps, 3 * heads, 128), generator=g).to(BF).cuda()
    status, size, gone = tb._int([0]), 0, 0
    for k in range(steps):
        new = x[k * chunk:(k + 1) * chunk]
        drop = max(0, size + chunk - window)
        api.page_free(kv, *s, first=tb._int([drop]), starts=starts, status=status)
        dropped = size if drop >= size else drop // page * page
        gone, size = gone + dropped, size - dropped
        slots, pos = api.page_append(kv, *s, tb._int([chunk]), chunk, starts=starts, status=status)
        size += chunk
        assert pos.tolist() == list(range(k * chunk, (k + 1) * chunk)) and gone + size == (k + 1) * chunk
        api.page_write(kv, new[:, heads:2 * heads], new[:, 2 * heads:], slots, rope=rope, positions=pos, status=status)
        q = api.rope(new[:, :heads], pos, rope)
        out = api.page_attention(q, kv, s[1], s[2], max_kv=192, status=status)
        alone = api.allocate_pages(12, heads, page, fmt)
        i = torch.arange(size).cuda()
        kept = x[gone:gone + size]
        api.page_write(alone, kept[:, heads:2 * heads], kept[:, 2 * heads:], i, rope=rope, positions=gone + i)
        table = torch.arange(12, dtype=torch.int32).view(1, 12).cuda()
        assert torch.equal(out, api.page_attention(q, alone, table, s[2], max_kv=192))
    assert gone > 0 and int(starts) == gone and int(status) == 0


def test_a_slide_is_captured_and_replayed():
    kv = tb._filled(40, 1, 16, I8, 3)
    s, m = tb._state(kv, 3, 10), Model(kv, 3, 10)
    starts = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert _append(kv, s, [100, 33, 0], starts) == m.append([100, 33, 0], 133)
    counts, drop = tb._int([32, 1, 5]), tb._int([32, 0, 0])

    def turn():
        api.page_free(kv, *s, first=drop, starts=starts)
        return api.page_append(kv, *s, counts, 38, starts=starts)

    def model():
        m.give(drop.tolist(), [0] * 3)
        return m.append(counts.tolist(), 38)[:2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn()
    torch.cuda.current_stream().wait_stream(side)
    model()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, pos = turn()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert (slots.tolist(), pos.tolist()) == model() and starts.tolist() == m.start
    m.check(kv, *s)


def test_refused_starts():
    kv = api.allocate_pages(8, 1, 16, BF)
    s = tb._state(kv, 2, 4)
    one, good = tb._int([0, 0]), torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (one, good[:1], good.cpu(), good.view(1, 2), torch.zeros(4, dtype=torch.int64, device="cuda")[::2]):
        for call in (lambda: api.page_append(kv, *s, one, 0, starts=bad), lambda: api.page_fork(kv, *s, one - 1, starts=bad),
                     lambda: api.page_free(kv, *s, last=one, starts=bad)):
            with pytest.raises(ValueError):
                call()
