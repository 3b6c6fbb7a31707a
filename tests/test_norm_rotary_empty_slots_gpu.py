"""Gradients of the head norms where teams of one warp have runs of different lengths: slots without a head take no part in the
weights' gradients, also with eps = 0, where the norm of nothing is not finite."""
import numpy as np
import pytest

from linear_attention_sequence_qkv_gb300 import gdn
from oracle import attention_ops as A
from test_norm_rotary_gpu import check, dev, make  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
# an odd number of tokens, runs that are no multiple of the heads in flight, parts that straddle q and k, wide and odd heads
@pytest.mark.parametrize("B,T,Hq,Hk,d,rot", [(1, 3, 3, 0, 64, 64), (1, 1, 1, 0, 64, 32), (1, 7, 5, 2, 128, 128), (3, 5, 1, 1, 32, 32),
                                             (1, 4999, 7, 3, 64, 64), (1, 3001, 3, 2, 128, 32), (1, 5, 2, 1, 256, 64), (1, 3, 2, 1, 7, 6)])
def test_without_eps(dev, B, T, Hq, Hk, d, rot, layout, dtype):  # noqa: F811
    s = make(dev, B, T, Hq, Hk, d, dtype)
    table, kw = gdn.rotary_table(rot, device=dev), dict(d=d, rot=rot, layout=layout, eps=0.0)
    got = gdn.norm_rotary(s["q"], s["k"], s["qw"], s["kw"], table, **kw)
    grads = gdn.norm_rotary_backward(s["q"], s["k"], s["qw"], s["kw"], table, s["gq"], s["gk"], **kw)
    check(s, got, grads, np.broadcast_to(np.arange(T), (B, T)), A.frequencies(rot), d, rot, layout, dtype, eps=0.0)
