"""The workspace of the window attention's backward (no GPU): partial sums for the sinks' later queries, of the sequences that have
any."""
import pytest

from linear_attention_sequence_qkv_gb300 import build, gdn


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


@pytest.mark.parametrize("N,window,sinks,mib", [(5000, 8192, 130, 512), (5000, 1024, 4, 100)])
def test_workspaces_of_long_packed_calls(lib, N, window, sinks, mib):
    """262144 tokens in 5000 sequences."""
    T = 262144
    desc = gdn.gdn_window_attention_desc_init(1, T, T, N if N > 1 else 0, 32, 16, 128, window, sinks, gdn.GDN_BF16)
    assert gdn.gdn_window_attention_backward_workspace_bytes(desc) <= mib << 20
