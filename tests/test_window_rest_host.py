"""The workspace of the window attention's backward (no GPU): partial sums for the sinks' later queries, of the sequences that have
any and of as many chunks as the GPU has use for."""
import pytest

from linear_attention_sequence_qkv_gb300 import build, gdn

CTAS = 8 * 152   # chunks' CTAs beyond which a chunk gets longer


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


@pytest.mark.parametrize("T,N,Hq,Hk,d,window,sinks", [
    (262144, 5000, 32, 16, 128, 1024, 4), (262144, 5000, 32, 16, 128, 8192, 130), (65536, 512, 32, 16, 128, 4096, 130),
    (65536, 512, 32, 8, 64, 100000, 64), (100000, 100000, 8, 8, 64, 1, 4), (131072, 1, 32, 16, 128, 128, 512),
    (131072, 1, 32, 16, 128, 128, 4096), (131072, 1, 32, 16, 128, 1024, 4096), (1 << 20, 1, 8, 1, 128, 4096, 1 << 20), (32768, 7, 8, 2, 200, 64, 2000)])
def test_partial_sums_are_bounded(lib, T, N, Hq, Hk, d, window, sinks):
    """A tile of sinks of a sequence that can have a rest has one own part and one chunk begun; all chunks together are CTAS more
    (rounded up for a head)."""
    desc = gdn.gdn_window_attention_desc_init(1, T, T, N if N > 1 else 0, Hq, Hk, d, window, sinks, gdn.GDN_BF16)
    tiles = min(-(-min(sinks, T) // 128), max(0, (T - window) // 128))
    tiles = min(tiles * min(N, T // (window + 128)), T // 128)   # of all sequences
    width = 64 if d <= 64 else 128 if d <= 128 else 256
    part = min(128, sinks) * 2 * width * 4
    most = (CTAS + Hk + Hk * tiles * 2) * part if tiles else 0
    tables = 256 * 8 + 4 * (3 * (N + 1) + tiles + 1) + 4 * T * Hq   # status, tables, delta
    assert gdn.gdn_window_attention_backward_workspace_bytes(desc) <= most + tables


@pytest.mark.parametrize("N,window,sinks,mib", [(5000, 8192, 130, 512), (5000, 1024, 4, 100), (1, 128, 4096, 512), (1, 1024, 4096, 512)])
def test_workspaces_of_long_packed_calls(lib, N, window, sinks, mib):
    """As numbers: 262144 tokens in 5000 sequences, 131072 in one."""
    T = 262144 if N > 1 else 131072
    desc = gdn.gdn_window_attention_desc_init(1, T, T, N if N > 1 else 0, 32, 16, 128, window, sinks, gdn.GDN_BF16)
    assert gdn.gdn_window_attention_backward_workspace_bytes(desc) <= mib << 20


def test_sizes_at_the_limits(lib):
    """The plan's own arithmetic at the largest sizes that a descriptor takes."""
    most = 2 ** 31 - 2 ** 16 - 1
    for B, Tq, Tk, packed, Hq, Hk, d, window, sinks in ((1, most, most, 0, 1, 1, 1, 1, 2 ** 31 - 1), (1, most, most, 70000, 64, 1, 8, 5, 2 ** 31 - 1),
                                                        (1, 0, most, 0, 1, 1, 1, 1, 4), (1, most, 0, 0, 1, 1, 1, 1, 4), (1, most, most, 0, 1000, 1, 1, 2 ** 31 - 1, 9)):
        desc = gdn.gdn_window_attention_desc_init(B, Tq, Tk, packed, Hq, Hk, d, window, sinks, gdn.GDN_BF16)
        assert gdn.gdn_window_attention_backward_workspace_bytes(desc) < 1 << 48
