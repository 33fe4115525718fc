"""What the calls return where no output tensor was given (rows that no sequence has,
and rows of sequences that were skipped, are zero and not leftovers), and what a
program learns of a step that its cache has no pages for."""
import pytest
import torch

from tests.test_gpu_decode import BAD, FULL, _filled, _ivc, dev

pytestmark = pytest.mark.gpu


def _leave_nans(*shape):
    """A freed block of this size that holds NaN: the next tensor of the size gets it."""
    torch.cuda.synchronize()
    x = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    del x


def test_rows_of_skipped_sequences_are_zero():
    ivc = _ivc()
    p = _filled(ivc, [40, 20], [6, 6])
    q = torch.randn(15, 4, 64, dtype=torch.bfloat16, device="cuda")
    off, seqs = dev([0, 6, 12]), dev([0, 7])          # there is no sequence 7
    ws = ivc.new_workspace(ivc.tree_attention_workspace_size(p.gpu, 15, 4, 2))
    good = ivc.tree_attention(p.gpu, 0, q, None, off, workspace=ws)
    for _ in range(3):
        _leave_nans(15, 4, 64)
        out = ivc.tree_attention(p.gpu, 0, q, None, off, seqs=seqs, workspace=ws)
        assert ivc.device_status(ws) == BAD
        assert torch.equal(out[:6], good[:6]) and (out[6:] == 0).all()


def test_rows_behind_the_last_sequence_are_zero():
    ivc = _ivc()
    p = _filled(ivc, [40, 20], [6, 6])
    x = torch.randn(15, 8 * 64, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    off, pos = dev([0, 6, 12]), dev(range(15))
    ws = ivc.new_workspace(256)
    for _ in range(3):
        _leave_nans(15, 4, 64)
        q = ivc.qk_norm_rope(p.gpu, 0, x, one, one, pos, off, workspace=ws)
        assert ivc.device_status(ws) == 0
        assert (q[:12] != 0).any(-1).all() and (q[12:] == 0).all()
        _leave_nans(15, 4, 64)
        out = ivc.tree_attention(p.gpu, 0, q, None, off)
        assert torch.isfinite(out).all() and (out[12:] == 0).all()


def test_a_step_without_enough_pages_is_told_by_the_status_word():
    """The whole step over one workspace: the bits say so, and the cache stays as it was."""
    ivc = _ivc()
    c = ivc.Cache.empty(1, 3, 1, 16, 64, 2, 4)
    ws = ivc.new_workspace(max(ivc.tree_attention_workspace_size(c, 14, 2, 2),
                               ivc.cache_workspace_size(c, 2, ivc.MAX_TREE)))
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(14, 4 * 64, dtype=torch.bfloat16, device="cuda")
    off, pos = dev([0, 7, 14]), dev(list(range(14, 21)) * 2)
    p = torch.full((14, 50), 0.02, device="cuda")

    def step():
        ivc.cache_reserve(c, dev([7, 7]), workspace=ws)
        q = ivc.qk_norm_rope(c, 0, x, one, one, pos, off, workspace=ws)
        out = ivc.tree_attention(c, 0, q, None, off, workspace=ws)
        path, m, t = ivc.verify_drafts(p, None, dev([3] * 14), None, off, torch.zeros(14, device="cuda"),
                                       torch.zeros(2, device="cuda"), workspace=ws)
        ivc.cache_compact(c, m, path, workspace=ws)
        return out, m

    ivc.cache_reserve(c, dev([14, 14]), workspace=ws)
    ivc.cache_compact(c, dev([14, 14]), workspace=ws)
    assert ivc.device_status(ws) == 0
    out, m = step()                          # a second page each, and one is left
    assert m.tolist() == [7, 7] and ivc.device_status(ws) == FULL | BAD
    assert (out == 0).all() and c.length.tolist() == [14, 14] and c.n_pages.tolist() == [1, 1]
    ivc.cache_free(c, dev([1]), workspace=ws)
    assert ivc.device_status(ws) == 0
    x, off, pos = x[:7], dev([0, 7, 7]), pos[:7].contiguous()
    ivc.cache_reserve(c, dev([7, 0]), workspace=ws)
    q = ivc.qk_norm_rope(c, 0, x, one, one, pos, off, workspace=ws)
    out = ivc.tree_attention(c, 0, q, None, off, workspace=ws)
    ivc.cache_compact(c, dev([7, 0]), workspace=ws)
    assert ivc.device_status(ws) == 0
    assert (out != 0).any(-1).all() and c.length.tolist() == [21, 0]
