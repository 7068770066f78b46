"""Which sparse_attention calls cut their queries over the SMs, and their results: a workspace is
needed exactly where pieces are joined."""
import pytest

from test_gpu_mxfp4 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Q,H,K", [(1, 128, 512), (1, 128, 1024), (1, 128, 1280), (2, 128, 640), (2, 128, 1280),
                                   (4, 128, 1024), (8, 128, 1280), (16, 128, 1280), (1, 64, 512), (4, 64, 640),
                                   (2, 32, 512)])
def test_few_long_queries_are_cut(gkr, Q, H, K):
    """Whole, each of these would take one pair of SMs for 8 to 20 chunks, while most of the others
    have nothing to do, and longer than a list of 2048 entries, which is cut."""
    assert gkr.sparse_attention_workspace(H, Q, K) > 0
    Case(gkr, Q, H, K, seed=Q + H + K).check(gkr)


@pytest.mark.parametrize("Q,H,K", [(1, 128, 128), (1, 128, 256), (64, 128, 1280), (128, 128, 2048), (76, 8, 640),
                                   (40, 16, 640), (32, 64, 1024)])
def test_short_or_many_queries_are_not(gkr, Q, H, K):
    assert gkr.sparse_attention_workspace(H, Q, K) == 0
