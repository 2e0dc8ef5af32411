"""GPU checks of what the calls on the pages of sequences do with tables and lengths that cannot be: the
sequence is left as it is, or its length cut, the others are served, and it is reported."""
import pytest
import torch

from tests import test_page_book_gpu as tb
from video_kv_cache_gb300 import api
from video_kv_cache_gb300 import build as qbuild
from video_kv_cache_gb300 import qvg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qbuild.build()
    qvg.load()
    torch.cuda.set_device(0)


def _four(rows, pages, seed):
    """Sequences of 20, 7, 33 and 0 tokens, the first of `rows` rows, against the model."""
    kv = tb._filled(pages, 1, 16, tb.I8, seed)
    s, m = tb._state(kv, rows, 8), tb.Model(kv, rows, 8)
    counts = [20, 7, 33] + [0] * (rows - 3)
    assert tb._append(kv, s, counts) == m.append(counts, 60)
    return kv, s, m


# few rows and pages, a cluster of CTAs, and more rows than shared memory has room for
SIZES = [(6, 40), (6, 40000), (1100, 40)]


@pytest.mark.parametrize("rows,pages", SIZES)
@pytest.mark.parametrize("entry", ["past", "negative", "free"])
@pytest.mark.parametrize("new", [1, 40])
def test_growth_behind_a_last_page_that_cannot_be(rows, pages, entry, new):
    # the second sequence's part-filled page is no page of the pool, or a free one
    kv, s, m = _four(rows, pages, 1)
    bad = {"past": pages, "negative": -2, "free": m.free_pages()[1]}[entry]
    s[1][1, 0] = bad
    counts = [new, new, new] + [0] * (rows - 3)
    want = m.append([new, 0, new] + [0] * (rows - 3), 2 * new)
    slots, pos, copies, status = tb._append(kv, s, counts)
    assert status == qvg.QVG_DEV_BAD_INDEX
    assert slots == want[0][:new] + [-1] * new + want[0][new:] and pos == want[1][:new] + [-1] * new + want[1][new:]
    assert copies == want[2]
    m.held[1] = [bad]
    m.check(kv, *s)


@pytest.mark.parametrize("rows,pages", SIZES)
@pytest.mark.parametrize("entry", ["past", "negative", "free"])
def test_forks_of_a_last_page_that_cannot_be(rows, pages, entry):
    kv, s, m = _four(rows, pages, 2)
    bad = {"past": pages, "negative": -2, "free": m.free_pages()[1]}[entry]
    s[1][0, 1] = bad
    parents = [-1, -1, -1, 0, 2] + [0] * (rows - 5)
    want = m.fork([-1, -1, -1, -1, 2] + [-1] * (rows - 5))
    copies, status = tb._fork(kv, s, parents)
    assert status == qvg.QVG_DEV_BAD_INDEX and copies == want[0]
    m.held[0][1] = bad
    m.check(kv, *s)


def test_whole_pages_that_cannot_be_are_shared_as_they_are():
    kv, s, m = _four(6, 40, 3)
    s[1][2, 0] = 40
    copies, status = tb._fork(kv, s, [-1, -1, -1, 2, -1, -1])
    assert status == qvg.QVG_DEV_BAD_INDEX and s[2].tolist() == [20, 7, 33, 33, 0, 0]
    assert s[1][3, :3].tolist() == [40, s[1][2, 1].item(), copies[1][3]]


def test_lengths_past_the_table_are_cut_where_nothing_is_given_up_too():
    kv, s, m = _four(6, 40, 4)
    table, refs = s[1].clone(), s[0].clone()
    s[2].copy_(tb._int([20, 129, 33, -4, 0, 128]))
    for kw in (dict(last=tb._int([0] * 6)), dict(first=tb._int([0] * 6)), dict(first=tb._int([0] * 6), last=tb._int([0] * 6))):
        lens, status = s[2].clone(), tb._int([0])
        api.page_free(kv, refs, table, lens, status=status, **kw)
        assert int(status) == qvg.QVG_DEV_BAD_INDEX and lens.tolist() == [20, 128, 33, 0, 0, 128]
        assert torch.equal(table, s[1]) and torch.equal(refs, s[0])
        status.zero_()
        api.page_free(kv, refs, table, lens, status=status, **kw)
        assert int(status) == 0
