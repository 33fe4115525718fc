"""Values at the ends of the decode calls' ranges are refused on the host (runs without
a GPU)."""
import pytest

from tests.test_decode_refusals import EINVAL, PTR, WS, _cache, _lib


@pytest.mark.parametrize("scale", [2.4e38, 3e38, 3.4e38])
def test_a_scale_that_overflows_in_log2_units_is_refused(scale):
    """scale * log2(e) would be infinite, and a score of 0 times that no number."""
    L, c = _lib(), _cache()
    need = L.ivc_tree_attention_workspace_size(c, 4, 16, 2)
    call = lambda x: L.ivc_tree_attention(c, 0, PTR, 16 * 128, 4, 16, x, None, PTR, None, 2, PTR, WS,  # noqa: E731
                                          need - 1, None)
    assert call(scale) == EINVAL
    assert call(2e38) == -3                  # allowed: the next check, the workspace's size, refuses


def test_device_status_reads_on_the_workspaces_device(monkeypatch):
    """With another device current: its stream is not behind the calls that set the bits."""
    import contextlib
    import types

    import torch

    import vlm_visual_token_b200 as ivc
    current, used = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    def status(ws, bits, stream):
        used.append((ws.value if hasattr(ws, "value") else ws, stream.value))
        bits._obj.value = 64
        return -5

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream=100 + current[0]))
    monkeypatch.setattr(ivc, "lib", lambda: types.SimpleNamespace(ivc_device_status=status))
    ws = types.SimpleNamespace(device=torch.device("cuda:1"), data_ptr=lambda: WS)
    assert ivc.device_status(ws) == 64
    assert used == [(WS, 101)] and current == [0]
