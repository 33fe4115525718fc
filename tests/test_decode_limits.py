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
