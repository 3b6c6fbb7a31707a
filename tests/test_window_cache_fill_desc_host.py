"""The cache's filling takes a whole descriptor (no GPU): the queries' part has no effect, but is checked as in the other calls."""
import ctypes
import math

import pytest

from linear_attention_sequence_qkv_gb300 import build, gdn
from test_layer_ops_host import FAKE, INVALID, UNSUPPORTED, WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def desc(**kw):
    d = gdn.gdn_window_attention_desc_init(2, 30, 30, 0, 4, 2, 64, 5, 2, gdn.GDN_BF16)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def write(lib, d):   # as far as its workspace, which is missing
    return lib.gdn_window_cache_write(ctypes.byref(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, None, 0, None)


@pytest.mark.parametrize("of_queries", [dict(Hq=2), dict(Hq=64, q_stride_t=64 * 64), dict(Tq=0), dict(Tq=1), dict(scale=3.0), dict(q_stride_b=0)])
def test_queries_have_no_effect(lib, of_queries):
    d, n = desc(**of_queries), ctypes.c_size_t(0)
    assert lib.gdn_window_cache_write_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == gdn.GDN_OK and n.value > 0
    assert write(lib, d) == WORKSPACE


@pytest.mark.parametrize("bad,status", [(dict(Hq=0), INVALID), (dict(Hq=3), UNSUPPORTED), (dict(Tq=-1), INVALID), (dict(Tq=2 ** 31 - 1), UNSUPPORTED),
                                        (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(q_stride_t=255), INVALID)])
def test_queries_are_checked(lib, bad, status):
    assert write(lib, desc(**bad)) == status
    n = ctypes.c_size_t(0)
    assert lib.gdn_window_cache_write_workspace_bytes(ctypes.byref(desc(**bad)), ctypes.byref(n)) == status


@pytest.mark.parametrize("bad,status", [(dict(Hk=0), INVALID), (dict(Tk=-1), INVALID), (dict(k_stride_t=127), INVALID), (dict(v_stride_b=-1), INVALID),
                                        (dict(slots=6), INVALID), (dict(window=0), INVALID), (dict(N=3), INVALID), (dict(d=300), UNSUPPORTED),
                                        (dict(Tk=2 ** 31 - 1), UNSUPPORTED), (dict(dtype=7), UNSUPPORTED)])
def test_keys_are(lib, bad, status):
    assert write(lib, desc(**bad)) == status
