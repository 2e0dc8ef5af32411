"""GPU checks of the calls on the pages of sequences against a model of lists: what each sequence holds,
how many name each page, what lies in it."""
import copy
import random

import pytest
import torch

from tests import pages_model as pm
from tests import pages4_model as m4
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu
BF, HF, E4, I8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8
FORMATS = [BF, HF, E4, I8, m4.E2M1, m4.INT4]
ALL = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


def _pools(kv):
    return [t.view(torch.uint8) for t in (kv.k, kv.v, kv.k_scale, kv.v_scale, kv.k_group, kv.v_group) if t is not None]


def _filled(pages, heads, page, fmt, seed):
    kv = api.allocate_pages(pages, heads, page, fmt)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in _pools(kv):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    return kv


def _int(x, shape=None):
    t = torch.tensor(x, dtype=torch.int32).cuda()
    return t if shape is None else t.view(shape)


class Model:
    """The state in lists, the pools' bytes on the CPU as [page][head][token][bytes of the row]."""

    def __init__(self, kv, rows, entries):
        self.page, self.entries = kv.page_tokens, entries
        self.refs, self.held, self.size = [0] * kv.n_pages, [[] for _ in range(rows)], [0] * rows
        self.pools = [self._rows(t, kv) for t in _pools(kv)]

    @staticmethod
    def _rows(t, kv):
        return t.reshape(kv.n_pages, kv.heads, kv.page_tokens, -1).cpu().clone()

    def free_pages(self):
        return [p for p, n in enumerate(self.refs) if n <= 0]

    def need(self, n):
        return -(-n // self.page)

    def copy_rows(self, src, dst, rows, to=None):
        for a, b in zip(self.pools, self.pools if to is None else to):
            b[dst, :, :rows] = a[src, :, :rows]

    def append(self, counts, total):
        free, at, places, status = self.free_pages(), 0, 0, 0
        slots, pos, copies = [], [], [[-1] * len(counts), [-1] * len(counts), [0] * len(counts)]
        given = []   # refs change only once everybody's copy is known
        old_refs = list(self.refs)
        for b, c in enumerate(counts):
            n = self.size[b]
            if c < 0:
                status |= qvg.QVG_DEV_BAD_INDEX
                c = 0
            if c == 0:
                continue
            if self.need(n + c) > self.entries:
                status |= qvg.QVG_DEV_NO_PAGES
                slots += [-1] * c
                pos += [-1] * c
                continue
            if len(slots) + c > total:
                status |= qvg.QVG_DEV_BAD_INDEX
                slots += [-1] * c
                pos += [-1] * c
                continue
            cow = n % self.page > 0 and old_refs[self.held[b][-1]] > 1
            want = self.need(n + c) - self.need(n) + cow
            if want and places + want > len(free):
                status |= qvg.QVG_DEV_NO_PAGES
                places += want
                slots += [-1] * c
                pos += [-1] * c
                continue
            mine = free[places:places + want]
            places += want
            if cow:
                src = self.held[b][-1]
                copies[0][b], copies[1][b], copies[2][b] = src, mine[0], n % self.page
                self.refs[src] -= 1
                self.held[b][-1] = mine[0]
                self.copy_rows(src, mine[0], n % self.page)
                given.append(mine[0])
                mine = mine[1:]
            self.held[b] += mine
            given += mine
            self.size[b] = n + c
            for t in range(n, n + c):
                slots.append(self.held[b][t // self.page] * self.page + t % self.page)
                pos.append(t)
        for p in given:
            self.refs[p] = 1
        pad = [-1] * (total - len(slots))
        return (slots + pad)[:total], (pos + pad)[:total], copies, status

    def fork(self, parents):
        free, places, status = self.free_pages(), 0, 0
        copies = [[-1] * len(parents), [-1] * len(parents), [0] * len(parents)]
        for b, p in enumerate(parents):
            if p < 0:
                continue
            if p >= len(parents) or parents[p] >= 0 or self.size[b] != 0:
                status |= qvg.QVG_DEV_BAD_INDEX
                continue
            full, rest = self.size[p] // self.page, self.size[p] % self.page
            if rest:
                places += 1
                if places > len(free):
                    status |= qvg.QVG_DEV_NO_PAGES
                    continue
            self.held[b], self.size[b] = self.held[p][:full], self.size[p]
            for x in self.held[b]:
                self.refs[x] += 1
            if rest:
                src, dst = self.held[p][full], free[places - 1]
                self.held[b].append(dst)
                self.refs[dst] = 1
                self.copy_rows(src, dst, rest)
                copies[0][b], copies[1][b], copies[2][b] = src, dst, rest
        return copies, status

    def give(self, first, last):
        for b in range(len(self.size)):
            f, l = max(first[b], 0), max(last[b], 0)
            z = self.size[b] - min(l, self.size[b])
            a = z if f >= z and (f or l) else f // self.page * self.page
            if not f and not l:
                continue
            keep = self.held[b][a // self.page:self.need(z)] if z > a else []
            for x in self.held[b]:
                self.refs[x] -= 1
            for x in keep:
                self.refs[x] += 1
            self.held[b], self.size[b] = keep, z - a

    def check(self, kv, refs, table, lens, rows_too=True):
        assert lens.tolist() == self.size and refs.tolist() == self.refs
        t = table.tolist()
        for b, held in enumerate(self.held):
            assert t[b][:len(held)] == held
        for got, want in zip(_pools(kv), self.pools):
            assert torch.equal(self._rows(got, kv), want)


def _state(kv, rows, entries):
    return (torch.zeros(kv.n_pages, dtype=torch.int32, device="cuda"),
            torch.full((rows, entries), -1, dtype=torch.int32, device="cuda"),
            torch.zeros(rows, dtype=torch.int32, device="cuda"))


def _append(kv, s, counts, total=None, **kw):
    status, copies = _int([0]), torch.empty((3, len(counts)), dtype=torch.int32, device="cuda")
    slots, pos = api.page_append(kv, *s, _int(counts), sum(counts) if total is None else total, copies=copies,
                                 status=status, **kw)
    return slots.tolist(), pos.tolist(), copies.tolist(), int(status)


def _fork(kv, s, parents, **kw):
    status = _int([0])
    copies = api.page_fork(kv, *s, _int(parents), status=status, **kw).tolist()
    lens = s[2].tolist()
    for b, p in enumerate(parents):  # the fourth row: whole pages shared
        assert copies[3][b] == -1 if p < 0 or copies[3][b] < 0 else copies[3][b] == lens[b] // kv.page_tokens
    return copies[:3], int(status)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,heads,pages,rows,entries", [(16, 3, 60, 7, 12), (32, 1, 30, 5, 6), (128, 2, 40, 9, 9),
                                                          (64, 1, 300, 40, 8)])
def test_many_steps_against_the_model(fmt, page, heads, pages, rows, entries):
    # sequences grow, fork, slide and end, or run out of pages and entries; everything is compared after each step
    r = random.Random(pages + rows)
    kv = _filled(pages, heads, page, fmt, rows)
    s = _state(kv, rows, entries)
    m = Model(kv, rows, entries)
    for step in range(25):
        kind = r.choice(["append", "append", "fork", "free", "free"])
        if kind == "append":
            counts = [r.choice([0, 1, 1, 2, page, r.randint(0, 3 * page)]) for _ in range(rows)]
            total = sum(counts) + r.choice([0, 0, 3])
            got = _append(kv, s, counts, total)
            want = m.append(counts, total)
        elif kind == "fork":
            parents = [-1] * rows
            old = [b for b in range(rows) if m.size[b]]
            for b in range(rows):
                if not m.size[b] and old and r.random() < 0.7:
                    parents[b] = r.choice(old)
            got, want = _fork(kv, s, parents), m.fork(parents)
        else:
            first = [r.choice([0, 0, 0, r.randint(0, 2 * page), ALL]) for _ in range(rows)]
            last = [r.choice([0, 0, 0, 1, r.randint(0, page), ALL]) for _ in range(rows)]
            which = r.choice(["both", "first", "last"])
            st = _int([0])
            api.page_free(kv, *s, first=_int(first) if which != "last" else None,
                          last=_int(last) if which != "first" else None, status=st)
            m.give(first if which != "last" else [0] * rows, last if which != "first" else [0] * rows)
            got, want = int(st), 0
        assert tuple(got) == tuple(want) if isinstance(got, tuple) else got == want, (step, kind)
        m.check(kv, *s)


@pytest.mark.parametrize("fmt", FORMATS)
def test_copies(fmt):
    heads, page = 3, 16
    kv, other = _filled(20, heads, page, fmt, 1), _filled(9, heads, page, fmt, 2)
    m, o = Model(kv, 1, 1), Model(other, 1, 1)
    src, dst, rows = [3, 5, 3, -1, 19, 7], [0, 1, 2, 4, -1, 8], [16, 0, 7, 3, 5, 1]
    api.page_copy(kv, _int(src), _int(dst), rows=_int(rows))
    for a, b, n in zip(src, dst, rows):
        if a >= 0 and b >= 0:
            m.copy_rows(a, b, n)
    for got, want in zip(_pools(kv), m.pools):
        assert torch.equal(m._rows(got, kv), want)
    api.page_copy(kv, _int([19, 0, 2]), _int([8, 3, 0]), out=other)
    for a, b in ((19, 8), (0, 3), (2, 0)):
        m.copy_rows(a, b, page, o.pools)
    status = _int([0])
    api.page_copy(kv, _int([20, 1, 4]), _int([1, 9, 5]), rows=_int([3, 3, 17]), out=other, status=status)
    m.copy_rows(4, 5, page, o.pools)  # rows past the page are cut
    assert int(status) == qvg.QVG_DEV_BAD_INDEX
    for got, want in zip(_pools(other), o.pools):
        assert torch.equal(m._rows(got, other), want)
    api.page_copy(kv, _int([]), _int([]))


@pytest.mark.parametrize("pages,rows", [(1, 1), (17, 3), (16384, 5), (16385, 70), (70000, 3), (150001, 1500)])
def test_the_lowest_pages_of_small_and_large_pools(pages, rows):
    # one thread's 16 pages, a tile, several tiles and CTAs; in order whatever the order of threads
    g = torch.Generator().manual_seed(pages)
    kv = api.allocate_pages(pages, 1, 16, I8)
    refs = torch.randint(0, 3, (pages,), generator=g).to(torch.int32)
    free = (refs == 0).nonzero()[:, 0].tolist()
    counts = [int(x) for x in torch.randint(0, max(1, 2 * 16 * len(free) // rows), (rows,), generator=g)]
    entries = max(1, max(-(-c // 16) for c in counts))
    s = (refs.cuda(), torch.full((rows, entries), -1, dtype=torch.int32, device="cuda"),
         torch.zeros(rows, dtype=torch.int32, device="cuda"))
    slots, pos, copies, status = _append(kv, s, counts)
    at, want_slots, want_pos, used, short = 0, [], [], 0, False
    for c in counts:
        n = -(-c // 16)
        if at + n <= len(free) or n == 0:
            want_slots += [free[at + t // 16] * 16 + t % 16 for t in range(c)]
            want_pos += list(range(c))
            used = at + n
        else:
            short = True
            want_slots += [-1] * c
            want_pos += [-1] * c
        at += n
    assert slots == want_slots and pos == want_pos and (status == qvg.QVG_DEV_NO_PAGES) == short
    now = refs.clone()
    now[free[:used]] = 1
    assert torch.equal(s[0].cpu(), now)
    # and packed: every page in use, in order
    live = int((now > 0).sum())
    out = api.allocate_pages(live, 1, 16, I8)
    table, new_refs, n = api.page_compact(kv, *s, out)
    assert int(n) == live and torch.equal(new_refs.cpu(), now[now > 0])
    place = (now > 0).cumsum(0) - 1
    old = s[1].cpu().long()
    assert torch.equal(table.cpu(), torch.where(old >= 0, place[old.clamp(min=0)], -1).to(torch.int32))


@pytest.mark.parametrize("fmt", FORMATS)
def test_compaction(fmt):
    heads, page, rows, entries = 2, 32, 6, 10
    kv = _filled(50, heads, page, fmt, 3)
    s = _state(kv, rows, entries)
    m = Model(kv, rows, entries)
    m.append([100, 40, 0, 300, 64, 1], 505)
    _append(kv, s, [100, 40, 0, 300, 64, 1])
    _fork(kv, s, [-1, -1, 3, -1, -1, -1])
    m.fork([-1, -1, 3, -1, -1, -1])
    drop = [0, ALL, 0, 0, 70, 0]
    api.page_free(kv, *s, first=_int(drop))
    m.give(drop, [0] * rows)
    m.check(kv, *s)
    live = [p for p, n in enumerate(m.refs) if n > 0]
    before = [t.clone() for t in s]
    out = _filled(len(live) + 3, heads, page, fmt, 4)
    o = Model(out, rows, entries)
    status = _int([0])
    table, refs, n = api.page_compact(kv, *s, out, status=status)
    assert int(n) == len(live) and int(status) == 0 and all(torch.equal(a, b) for a, b in zip(s, before))
    for new, old in enumerate(live):
        m.copy_rows(old, new, page, o.pools)
    for got, want in zip(_pools(out), o.pools):
        assert torch.equal(m._rows(got, out), want)
    assert refs.tolist() == [m.refs[p] for p in live] + [0] * 3
    want = [[live.index(p) for p in held] + [-1] * (entries - len(held)) for held in m.held]
    assert table.tolist() == want
    # no room for the last two pages: their entries are left out, and it is reported
    small = api.allocate_pages(len(live) - 2, heads, page, fmt)
    table, refs, n = api.page_compact(kv, *s, small, status=status)
    assert int(n) == len(live) and int(status) == qvg.QVG_DEV_NO_PAGES
    assert table.tolist() == [[x if x < len(live) - 2 else -1 for x in row] for row in want]
    assert refs.tolist() == [m.refs[p] for p in live[:-2]]
    for got, w in zip(_pools(small), o.pools):
        assert torch.equal(m._rows(got, small), w[:len(live) - 2])
    # entries of nowhere and of free pages
    bad = s[1].clone()
    bad[0, 0], bad[3, 1] = 50, m.free_pages()[0]
    status.zero_()
    table, _, _ = api.page_compact(kv, s[0], bad, s[2], out, status=status)
    assert int(status) == qvg.QVG_DEV_BAD_INDEX and table[0, 0] == -1 and table[3, 1] == -1
    assert table[0, 1] == want[0][1]


def test_a_shared_last_page_is_copied_before_it_is_written():
    # two forks cut back into a page that they share: whoever grows gets a page of its own
    kv = _filled(12, 2, 16, E4, 5)
    s, m = _state(kv, 3, 4), Model(kv, 3, 4)
    assert _append(kv, s, [40, 0, 0]) == m.append([40, 0, 0], 40)
    assert _fork(kv, s, [-1, 0, 0]) == m.fork([-1, 0, 0])
    drop = [0, 13, 13]   # 27 tokens: 11 rows of a page of which the parent holds all 16
    api.page_free(kv, *s, last=_int(drop))
    m.give([0] * 3, drop)
    got, want = _append(kv, s, [0, 3, 0]), m.append([0, 3, 0], 3)
    assert got == want and got[2][0][1] == m.held[0][1] and got[2][2][1] == 11
    m.check(kv, *s)
    got, want = _append(kv, s, [1, 0, 20]), m.append([1, 0, 20], 21)
    assert got == want and got[2][0][2] == m.held[0][1]
    m.check(kv, *s)
    # nobody shares it now, and all at once
    assert _append(kv, s, [1, 1, 1]) == m.append([1, 1, 1], 3)
    m.check(kv, *s)


def test_sharers_that_grow_in_one_call():
    kv = _filled(20, 1, 16, m4.INT4, 6)
    s, m = _state(kv, 4, 4), Model(kv, 4, 4)
    assert _append(kv, s, [32, 0, 0, 0]) == m.append([32, 0, 0, 0], 32)
    assert _fork(kv, s, [-1, 0, 0, 0]) == m.fork([-1, 0, 0, 0])
    api.page_free(kv, *s, last=_int([5, 5, 5, 5]))
    m.give([0] * 4, [5] * 4)
    got, want = _append(kv, s, [1, 1, 1, 1]), m.append([1, 1, 1, 1], 4)
    assert got == want and m.refs[1] == 0   # each with a copy of its own, the page itself is free
    m.check(kv, *s)


@pytest.mark.parametrize("rows,pages", [(1024, 3000), (1025, 3000), (2500, 40000)])
def test_many_sequences(rows, pages):
    # more than a CTA's threads and than shared memory has room for, in one CTA and in a cluster of them
    kv = _filled(pages, 1, 16, I8, rows)
    s, m = _state(kv, rows, 3), Model(kv, rows, 3)
    r = random.Random(rows)
    counts = [r.randint(0, 40) if b % 3 == 0 else 0 for b in range(rows)]
    assert _append(kv, s, counts) == m.append(counts, sum(counts))
    parents = [b // 3 * 3 if b % 3 else -1 for b in range(rows)]
    assert _fork(kv, s, parents) == m.fork(parents)
    counts = [r.randint(0, 20) for b in range(rows)]
    assert _append(kv, s, counts) == m.append(counts, sum(counts))
    m.check(kv, *s)
    # all cut back to the prompts' first rows, many into a page that they share: whoever grows copies it
    drop = [max(0, n - 13) for n in m.size]
    api.page_free(kv, *s, last=_int(drop))
    m.give([0] * rows, drop)
    for counts in ([1 if b % 5 == 0 else 0 for b in range(rows)], [b % 3 for b in range(rows)]):
        got, want = _append(kv, s, counts), m.append(counts, sum(counts))
        assert got == want
    m.check(kv, *s)


def test_what_cannot_be_done_is_left_and_reported():
    kv = _filled(6, 1, 16, HF, 7)
    s, m = _state(kv, 4, 3), Model(kv, 4, 3)
    assert _append(kv, s, [20, 0, 0, 0]) == m.append([20, 0, 0, 0], 20)
    # past the row, too few pages from the second on (the fourth wants none of the row's end), bad counts
    for counts, total in (([40, 0, 0, 0], 40), ([1, 49, 1, 0], 51), ([1, 48, 40, 1], 90), ([-3, 5, 0, 0], 5),
                          ([1, 30, 16, 0], 31), ([3, 3, 3, 3], 0)):
        t, mm, ss = copy.deepcopy(kv), copy.deepcopy(m), tuple(x.clone() for x in s)
        got, want = _append(t, ss, counts, total), mm.append(counts, total)
        assert got == want and got[3], counts
        mm.check(t, *ss)
    status = _int([0])
    # lengths that cannot be: left alone
    odd = (s[0].clone(), s[1].clone(), _int([20, -1, 49, 0]))
    slots, _ = api.page_append(kv, *odd, _int([1, 1, 1, 1]), 4, status=status)
    assert int(status) == qvg.QVG_DEV_BAD_INDEX and slots.tolist()[1:3] == [-1, -1] and slots.tolist()[0] >= 0
    assert odd[2].tolist() == [21, -1, 49, 1]
    # forks of nobody, of oneself, of a fork, into a sequence that is not empty
    for parents in ([-1, 4, -1, -1], [-1, 1, -1, -1], [-1, 0, 1, -1], [1, -1, -1, -1]):
        t, mm, ss = copy.deepcopy(kv), copy.deepcopy(m), tuple(x.clone() for x in s)
        got, want = _fork(t, ss, parents), mm.fork(parents)
        assert got == want and got[1] == qvg.QVG_DEV_BAD_INDEX, parents
        mm.check(t, *ss)
    # more forks than free pages: the first ones get them
    refs = _int([1, 1, 1, 1, 0, 1])
    ss = (refs, s[1].clone(), s[2].clone())
    got = _fork(kv, ss, [-1, 0, 0, 0])
    assert got[1] == qvg.QVG_DEV_NO_PAGES and ss[2].tolist() == [20, 20, 0, 0] and ss[0].tolist() == [2, 1, 1, 1, 1, 1]
    # entries of nowhere and pages that are free already
    bad = s[1].clone()
    bad[0, 1] = 77
    ss = (s[0].clone(), bad, s[2].clone())
    status.zero_()
    api.page_free(kv, *ss, last=_int([ALL, 0, 0, 0]), status=status)
    assert int(status) == qvg.QVG_DEV_BAD_INDEX and ss[0].tolist()[0] == 0 and ss[2].tolist() == [0] * 4
    ss = (torch.zeros_like(s[0]), s[1].clone(), s[2].clone())
    status.zero_()
    api.page_free(kv, *ss, first=_int([ALL, -1, 0, 0]), status=status)
    assert int(status) == qvg.QVG_DEV_BAD_INDEX and not ss[0].any()


def test_capture_replay_other_streams_and_layers():
    # fork, grow and end, captured once and replayed; a second layer follows by the copies
    heads, page = 2, 16
    layers = [_filled(64, heads, page, fmt, 8) for fmt in (E4, BF)]
    s, m = _state(layers[0], 6, 8), Model(layers[0], 6, 8)
    m2 = Model(layers[1], 6, 8)
    _append(layers[0], s, [50, 0, 0, 7, 0, 0])
    m.append([50, 0, 0, 7, 0, 0], 57)
    parents, counts, drop = _int([-1, 0, 0, -1, 3, 3]), _int([0, 3, 3, 0, 3, 3]), _int([0, ALL, ALL, 0, ALL, ALL])

    def turn(stream=None):
        api.page_free(layers[0], *s, last=drop, stream=stream)
        copies = api.page_fork(layers[0], *s, parents, stream=stream)
        api.page_copy(layers[1], copies[0], copies[1], rows=copies[2], stream=stream)
        return api.page_append(layers[0], *s, counts, 12, stream=stream)

    def model():
        m.give([0] * 6, drop.tolist())
        src, dst, rows = m.fork(parents.tolist())[0]
        for a, b, n in zip(src, dst, rows):
            if a >= 0:
                m2.copy_rows(a, b, n)
        return m.append(counts.tolist(), 12)[:2]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots, pos = turn(side)
    torch.cuda.current_stream().wait_stream(side)
    assert (slots.tolist(), pos.tolist()) == model()
    with torch.cuda.stream(side):
        turn()
    torch.cuda.current_stream().wait_stream(side)
    model()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, pos = turn()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert (slots.tolist(), pos.tolist()) == model()
        m.check(layers[0], *s)
        for got, want in zip(_pools(layers[1]), m2.pools):
            assert torch.equal(m2._rows(got, layers[1]), want)


def test_a_cluster_of_ctas_is_captured_and_replayed():
    kv = api.allocate_pages(100000, 1, 16, I8)
    g = torch.Generator().manual_seed(3)
    start = torch.randint(0, 2, (kv.n_pages,), generator=g).to(torch.int32)
    refs, table, lens = start.cuda(), torch.full((3, 4000), -1, dtype=torch.int32, device="cuda"), _int([0, 0, 0])
    counts, total = _int([60000, 1, 17]), 60018
    api.page_append(kv, refs, table, lens, counts, total)   # (once before, as a capture wants)
    want = [t.clone() for t in (refs, table, lens)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, _ = api.page_append(kv, refs, table, lens, counts, total)
    free = (start == 0).nonzero()[:, 0]
    for _ in range(3):
        for t, v in ((refs, start.cuda()), (table, torch.full_like(table, -1)), (lens, torch.zeros_like(lens))):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((refs, table, lens), want))
        i = torch.arange(60000)
        assert torch.equal(slots[:60000].cpu(), free[i // 16] * 16 + i % 16) and int(slots[60000]) == int(free[3750]) * 16


@pytest.mark.parametrize("fmt", [BF, E4, m4.E2M1])
def test_sampling_continuations_end_to_end(fmt):
    # a prompt is written, forked, each fork grows by tokens of its own and attends; then old tokens are
    # dropped, and the cache is packed into a smaller one: attention is as over separate caches
    heads, page, n = 2, 16, 50
    g = torch.Generator().manual_seed(9)
    kv = api.allocate_pages(40, heads, page, fmt)
    s = _state(kv, 3, 8)
    rows = torch.randn((n + 9, 2 * heads, 128), generator=g).to(BF).cuda()
    status = _int([0])
    slots, pos = api.page_append(kv, *s, _int([n, 0, 0]), n, status=status)
    api.page_write(kv, rows[:n, :heads], rows[:n, heads:], slots, status=status)
    api.page_fork(kv, *s, _int([-1, 0, 0]), status=status)
    slots, pos = api.page_append(kv, *s, _int([2, 3, 4]), 9, status=status)
    api.page_write(kv, rows[n:, :heads], rows[n:, heads:], slots, status=status)
    assert pos.tolist() == [50, 51, 50, 51, 52, 50, 51, 52, 53] and s[2].tolist() == [52, 53, 54]
    # the same three sequences, each in pages of its own
    alone = api.allocate_pages(12, heads, page, fmt)
    table = torch.arange(12, dtype=torch.int32).view(3, 4).cuda()
    for b, (first, count) in enumerate(((0, 2), (2, 3), (5, 4))):
        x = torch.cat([rows[:n], rows[n + first:n + first + count]])
        i = torch.arange(n + count).cuda()
        api.page_write(alone, x[:, :heads], x[:, heads:], table[b, i // page].long() * page + i % page)
    Q = torch.randn((3, 4, 128), generator=g).to(BF).cuda()
    want = api.page_attention(Q, alone, table, s[2], max_kv=64)
    assert torch.equal(api.page_attention(Q, kv, s[1], s[2], max_kv=64), want)
    out = api.allocate_pages(9, heads, page, fmt)
    packed, refs, live = api.page_compact(kv, *s, out, status=status)
    assert int(live) == 6  # three shared, and one of each
    assert torch.equal(api.page_attention(Q, out, packed, s[2], max_kv=64), want)
    # two pages of old tokens go: the rest attends as a shorter sequence
    api.page_free(kv, *s, first=_int([33, 33, 33]), status=status)
    assert s[2].tolist() == [20, 21, 22] and int(status) == 0
    short = torch.cat([table[:, 2:], table[:, :2]], 1).contiguous()
    assert torch.equal(api.page_attention(Q, kv, s[1], s[2], max_kv=64),
                       api.page_attention(Q, alone, short, s[2], max_kv=64))
    api.page_free(kv, *s, last=_int([ALL] * 3), status=status)
    assert not s[0].any() and bool((s[1] == -1).all()) and int(status) == 0


def test_refused_arguments():
    kv = api.allocate_pages(8, 1, 16, BF)
    s = _state(kv, 2, 4)
    one = _int([0, 0])
    bad = [
        lambda: api.page_append(kv, s[0][:7], s[1], s[2], one, 0),
        lambda: api.page_append(kv, s[0].long(), s[1], s[2], one, 0),
        lambda: api.page_append(kv, s[0], s[1], s[2], one.cpu(), 0),
        lambda: api.page_append(kv, s[0], s[1], s[2], _int([0]), 0),
        lambda: api.page_append(kv, s[0], s[1], s[2], one, -1),
        lambda: api.page_append(kv, s[0], s[1][:, ::2], s[2], one, 0),
        lambda: api.page_append(kv, s[0], s[1], s[2], one, 0, copies=one),
        lambda: api.page_fork(kv, s[0], s[1], s[2], one.float()),
        lambda: api.page_fork(kv, s[0], s[1], s[2][:1], one),
        lambda: api.page_fork(kv, s[0], s[1], s[2], one, status=torch.zeros(1, dtype=torch.int32)),
        lambda: api.page_free(kv, *s),
        lambda: api.page_free(kv, *s, first=_int([1])),
        lambda: api.page_copy(kv, one, _int([0])),
        lambda: api.page_copy(kv, one.view(1, 2), one),
        lambda: api.page_copy(kv, one, one, out=api.allocate_pages(8, 2, 16, BF)),
        lambda: api.page_copy(kv, one, one, out=api.allocate_pages(8, 1, 16, HF)),
        lambda: api.page_compact(kv, *s, api.allocate_pages(8, 1, 32, BF)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qvg.QVGError):  # into itself
        api.page_compact(kv, *s, kv)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    many = _state(kv, 1025, 4)  # the wants of up to 1024 sequences need no workspace
    none = torch.full((1025,), -1, dtype=torch.int32, device="cuda")
    for call in (lambda: api.page_append(kv, *many, none, 0, workspace=small), lambda: api.page_fork(kv, *many, none, workspace=small),
                 lambda: api.page_compact(kv, *s, api.allocate_pages(2, 1, 16, BF), workspace=small)):
        with pytest.raises(qvg.QVGError) as e:
            call()
        assert e.value.code == qvg.QVG_ERR_WORKSPACE


def test_numbers_in_the_place_of_vectors_are_refused():
    kv = api.allocate_pages(8, 1, 16, BF)
    refs, table, lens = _state(kv, 1, 4)
    for args in ((refs, table, lens[0]), (lens[0], table, lens), (refs, lens[0], lens), (refs, table[0], lens)):
        with pytest.raises(ValueError):
            api.page_free(kv, *args, last=_int([ALL]))
