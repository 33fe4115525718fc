"""Cache operations whose device data are wrong change nothing at all, wherever the
wrong entry stands."""
import numpy as np
import pytest
import torch

from tests.test_gpu_decode import BAD, Pair, _ivc, dev

pytestmark = pytest.mark.gpu
TENSORS = ("k", "v", "table", "length", "n_pages", "ref", "free_list", "free_count")


def _refused(p, call):
    """The call sets IVC_DEV_BAD_CACHE and leaves every tensor of the cache as it was."""
    before = [getattr(p.gpu, x).clone() for x in TENSORS]
    call()
    assert p.ivc.device_status(p.ws) == BAD
    for name, was in zip(TENSORS, before):
        assert torch.equal(getattr(p.gpu, name), was), name


def _batch(**kw):
    """Sequences 0, 1, 2 of 40, 20 and 50 tokens, and 3 that shares 0's full pages."""
    p = Pair(_ivc(), **kw)
    p.reserve([40, 20, 50], [0, 1, 2])
    p.compact([40, 20, 50], seqs=[0, 1, 2])
    p.fork([0], [3], True)
    return p


def _table(seq, page, value):
    def change(c):
        c.table[seq, page] = value
    return change


def _nobodys(c):
    c.ref[int(c.table[2, 3])] = 0


def _two_holders_counted_as_one(c):
    c.table[1, 1] = c.table[2, 3]


def _twice_in_one_sequence(c):
    c.table[2, 3] = c.table[2, 2]


def _list_without_room(c):
    c.free_count[0] = 62                     # 10 pages are held of 64


@pytest.mark.parametrize("change", [
    _table(2, 3, -1), _table(2, 3, 64), _table(2, 3, 1 << 30), _nobodys, _two_holders_counted_as_one,
    _twice_in_one_sequence, _list_without_room])
@pytest.mark.parametrize("what", ["free", "compact", "compact with a keep list"])
def test_pages_that_cannot_be_given_back(what, change):
    """Every page of sequences 0, 1, 3 and 2 is given back but for those kept: a wrong
    one behind sound ones."""
    p = _batch()
    change(p.gpu)
    order = [0, 1, 3, 2]
    if what == "free":
        _refused(p, lambda: p.ivc.cache_free(p.gpu, dev(order), workspace=p.ws))
    elif what == "compact":
        _refused(p, lambda: p.ivc.cache_compact(p.gpu, dev([0] * 4), None, dev([0] * 4), dev(order),
                                                workspace=p.ws))
    else:                                    # sequence 1 and 2 keep two tokens that move
        if change is _list_without_room:
            p.gpu.free_count[0] = 63
        _refused(p, lambda: p.ivc.cache_compact(p.gpu, dev([0, 2, 0, 2]), dev([[0, 0], [1, 3], [0, 0], [2, 9]]),
                                                dev([0] * 4), dev(order), workspace=p.ws))


def _entry(value):
    def change(c):
        c.free_list[int(c.free_count) - 2] = value
    return change


def _held(c):
    _entry(int(c.table[0, 0]))(c)


def _twice(c):
    _entry(int(c.free_list[int(c.free_count) - 1]))(c)


@pytest.mark.parametrize("change", [_entry(-1), _entry(64), _entry(1 << 30), _held, _twice])
@pytest.mark.parametrize("what", ["reserve one", "reserve several", "fork", "fork shared"])
def test_pages_that_cannot_be_taken(what, change):
    """The second page from the top of the free list is none, held, or there twice."""
    p = _batch()
    change(p.gpu)
    call = {"reserve one": lambda: p.ivc.cache_reserve(p.gpu, dev([48]), dev([5]), workspace=p.ws),
            "reserve several": lambda: p.ivc.cache_reserve(p.gpu, dev([3, 10, 16]), dev([5, 6, 7]),
                                                           workspace=p.ws),
            "fork": lambda: p.ivc.cache_fork(p.gpu, dev([2]), dev([5]), False, workspace=p.ws),
            "fork shared": lambda: p.ivc.cache_fork(p.gpu, dev([0, 1]), dev([6, 5]), True, workspace=p.ws)}
    _refused(p, call[what])


def test_a_wrong_entry_that_is_not_touched_does_not_matter():
    """The third entry from the top: a call that takes two pages is right, the next is refused."""
    p = _batch()
    at = int(p.gpu.free_count) - 3
    was = int(p.gpu.free_list[at])
    p.gpu.free_list[at] = 1 << 30
    p.ivc.cache_reserve(p.gpu, dev([20]), dev([5]), workspace=p.ws)
    assert p.ivc.device_status(p.ws) == 0
    _refused(p, lambda: p.ivc.cache_reserve(p.gpu, dev([20]), dev([6]), workspace=p.ws))
    p.gpu.free_list[at] = was
    p.ref.reserve([20], [5])
    p.same()
    p.reserve([20], [6])
    p.free([5, 6, 0, 3])


def test_a_wrong_entry_behind_many_sequences():
    """More sequences than a CTA has threads, the wrong page in the last ones."""
    n, pt = 1500, 16
    p = Pair(_ivc(), layers=1, pages=4 * n, kv_heads=1, pt=pt, seqs=2 * n, max_pages=3)
    p.ws = p.ivc.new_workspace(p.ivc.cache_workspace_size(p.gpu, n, 0))
    lens = np.random.RandomState(0).randint(1, 3 * pt, n).tolist()
    lens[-1] = 3 * pt
    seqs, rest = list(range(n)), list(range(n, 2 * n))
    p.reserve(lens, seqs)
    p.compact(lens, seqs=seqs)
    good = int(p.gpu.table[n - 1, 2])
    p.gpu.table[n - 1, 2] = 4 * n
    _refused(p, lambda: p.ivc.cache_free(p.gpu, dev(seqs), workspace=p.ws))
    _refused(p, lambda: p.ivc.cache_compact(p.gpu, dev([0] * n), None, dev([0] * n), dev(seqs), workspace=p.ws))
    p.gpu.table[n - 1, 2] = good
    at = int(p.gpu.free_count) - n
    entry = int(p.gpu.free_list[at])
    p.gpu.free_list[at] = good               # the n-th page taken is another's
    _refused(p, lambda: p.ivc.cache_reserve(p.gpu, dev([1] * n), dev(rest), workspace=p.ws))
    _refused(p, lambda: p.ivc.cache_fork(p.gpu, dev(seqs), dev(rest), False, workspace=p.ws))
    p.gpu.free_list[at] = entry
    p.same()
    p.free(seqs)
