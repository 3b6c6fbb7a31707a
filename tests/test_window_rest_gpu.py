"""The sinks' queries beyond the window in the window attention's backward: many tiles of sinks, packed sequences of which only
some have such queries."""
import numpy as np
import pytest
import torch

from linear_attention_sequence_qkv_gb300 import gdn
from test_window_attention_gpu import ACT, check, dev, make  # noqa: F401

pytestmark = pytest.mark.gpu


def both(q, k, v, dout, kw):
    f = gdn.window_attention_forward(q, k, v, **kw)
    g = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    assert gdn.gdn_device_status(g.workspace) == gdn.GDN_OK
    again = gdn.window_attention_backward(q, k, v, f.out, f.lse, dout, **kw)
    assert all(torch.equal(getattr(g, n), getattr(again, n)) for n in ("dq", "dk", "dv"))
    return f, g


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,Tq,Tk,Hq,Hk,d,window,sinks", [(2, 1500, 1500, 4, 2, 64, 40, 700), (1, 1000, 1700, 2, 2, 128, 300, 5000),
                                                          (1, 1300, 900, 3, 1, 64, 1, 257), (3, 1281, 1281, 2, 1, 128, 640, 512)])
def test_many_tiles_of_sinks(dev, B, Tq, Tk, Hq, Hk, d, window, sinks, dtype):  # noqa: F811
    q, k, v, dout = make(dev, B, Tq, Tk, Hq, Hk, d, dtype)
    f, g = both(q, k, v, dout, dict(d=d, window=window, sinks=sinks))
    check(q, k, v, dout, f, g, [(b, 0, Tq, 0, Tk) for b in range(B)], d, window, sinks, f.desc.scale, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lengths,keys", [([900, 0, 30, 1300, 129, 1, 500], None), ([100, 5, 700, 0, 300], [900, 700, 700, 600, 100]),
                                          ([1, 2, 3, 4, 5] * 250 + [1000] + [3] * 1200 + [700], None), ([40] * 60, None), ([800], None)])
@pytest.mark.parametrize("Hq,Hk,d,window,sinks", [(4, 2, 64, 50, 300), (3, 1, 128, 130, 4)])
def test_packed_sequences_with_and_without(dev, lengths, keys, Hq, Hk, d, window, sinks, dtype):  # noqa: F811
    keys_ = keys or lengths
    cuq, cuk = ([0] + np.cumsum(x).tolist() for x in (lengths, keys_))
    q, k, v, dout = make(dev, 1, cuq[-1], cuk[-1], Hq, Hk, d, dtype)
    kw = dict(d=d, window=window, sinks=sinks, cu_seqlens=torch.tensor(cuq, dtype=torch.int32, device=dev),
              cu_seqlens_k=torch.tensor(cuk, dtype=torch.int32, device=dev) if keys else None)
    f, g = both(q, k, v, dout, kw)
    some = sorted(range(len(lengths)), key=lambda n: -lengths[n])[:6] + list(range(0, len(lengths), 300))
    check(q, k, v, dout, f, g, [(0, cuq[n], lengths[n], cuk[n], keys_[n]) for n in sorted(set(some))], d, window, sinks, f.desc.scale, dtype)
