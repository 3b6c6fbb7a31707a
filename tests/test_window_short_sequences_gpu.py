"""Gradients of the window attention's short sequences: a query that sees one key has none for q and k, exactly; and where a few
keys share the weight, dP - delta cancels, so that delta is not to come from the rounded output."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import gdn
from oracle import attention_ops as A
from test_window_attention_gpu import ACT, dev, make, n64  # noqa: F401

pytestmark = pytest.mark.gpu


def both(q, k, v, dout, kw):
    f = gdn.window_attention_forward(q, k, v, **kw)
    return f, gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,T,Hq,Hk,d,window", [(1, 1, 1, 1, 64, 16), (3, 1, 4, 2, 128, 1), (2, 1, 3, 1, 96, 1000), (2, 200, 4, 2, 128, 1), (1, 300, 3, 1, 64, 1),
                                                (1, 70, 2, 2, 40, 1), (2, 50, 2, 1, 33, 1)])
def test_one_key(dev, B, T, Hq, Hk, d, window, dtype):  # noqa: F811
    q, k, v, dout = make(dev, B, T, T, Hq, Hk, d, dtype)
    f, g = both(q, k, v, dout, dict(d=d, window=window, sinks=0))
    assert torch.equal(f.out.view(B, T, Hk, -1, d), v.reshape(B, T, Hk, 1, d).expand(B, T, Hk, Hq // Hk, d))
    assert not g.dq.any() and not g.dk.any()
    want = n64(dout).reshape(B, T, Hk, -1, d).sum(3).reshape(B, T, -1)   # P is 1 up to a few of fp32's roundings
    assert (np.abs(n64(g.dv) - want) <= A.bound(want, 2.0 ** -18 * np.abs(n64(dout)).reshape(B, T, Hk, -1, d).sum(3).reshape(B, T, -1), dtype)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_first_queries_of_sequences(dev, dtype):  # noqa: F811
    """dq of a sequence's first query is 0 whatever follows, with queries that follow a past it is not the first any more."""
    lengths, keys = [1, 5, 1, 140, 1, 2], [1, 5, 4, 140, 0, 1]
    cuq, cuk = ([0] + np.cumsum(x).tolist() for x in (lengths, keys))
    q, k, v, dout = make(dev, 1, cuq[-1], cuk[-1], 4, 2, 64, dtype)
    cu = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    f, g = both(q, k, v, dout, dict(d=64, window=30, sinks=1, cu_seqlens=cu(cuq), cu_seqlens_k=cu(cuk)))
    zero = [cuq[0], cuq[1], cuq[3], cuq[4], cuq[5], cuq[5] + 1]   # sees one key, or none
    some = [t for t in range(cuq[-1]) if t not in zero]
    assert not g.dq[0, zero].any() and bool(g.dq[0, some].any(-1).all())
    assert not g.dk[0, cuk[0]].any() and not g.dk[0, cuk[5]].any()
