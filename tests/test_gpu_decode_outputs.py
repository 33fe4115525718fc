"""What the calls return where no output tensor was given: rows that no sequence
has, and rows of sequences that were skipped, are zero and not leftovers."""
import pytest
import torch

from tests.test_gpu_decode import BAD, _filled, _ivc, dev

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
