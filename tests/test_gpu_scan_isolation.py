"""Infinite and undefined values stay where the definition has them: documents of
a packed row do not see each other's, also where the time axis is cut between
them.  Equal bits are asked for, so no tolerance is needed."""
import pytest
import torch

import dsc_inputs as di
from tests import gpu_util as gu
from tests.test_gpu_scan import BF16, F32, dev, make

pytestmark = pytest.mark.gpu

TOKENS = ("x", "delta", "Bm", "Cm", "z")


@pytest.fixture(scope="module")
def dsc():
    import dynamic_short_causal_amd as d
    return d


def two_documents(B, T, cut):
    one = torch.cat([torch.arange(cut), torch.arange(T - cut)]).to(torch.int32)
    return one.repeat(B, 1).to(gu.dev())


# backward chunks of one tile (16 or 8 tokens), forward chunks of 64 tokens: the
# boundary lies in the middle of a chunk, chunks away from most of either document
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("N,W,dtype", [(16, 4, F32), (3, 4, BF16), (8, 2, F32), (24, 8, BF16),
                                       (64, 4, BF16)])
def test_a_later_document_does_not_reach_back(dsc, N, W, dtype, bad):
    B, T, cut = 1, 700, 333
    p = dev(make(B, T, 64, N, W, 1, dtype, 2000 + N))
    p["dy"] = di.randn((B, T, 64), 1.0, 2100, "bf16" if dtype == BF16 else "f32").to(gu.dev())
    pos = two_documents(B, T, cut)
    want = dsc.scan_bwd(**p, act=True, pos=pos)
    for name in TOKENS + ("dy",):
        q = dict(p, **{name: p[name].clone()})
        q[name][:, cut:] = bad
        got = dsc.scan_bwd(**q, act=True, pos=pos)
        for k in ("dx", "ddelta", "dz", "dBm", "dCm"):
            assert torch.equal(got[k][:, :cut], want[k][:, :cut]), (name, k)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("N,W,dtype", [(16, 4, F32), (3, 4, BF16), (8, 2, F32), (24, 8, BF16),
                                       (64, 4, BF16)])
def test_an_earlier_document_does_not_reach_on(dsc, N, W, dtype, bad):
    B, T, cut = 1, 700, 333
    p = dev(make(B, T, 64, N, W, 1, dtype, 2200 + N))
    p["dy"] = di.randn((B, T, 64), 1.0, 2300, "bf16" if dtype == BF16 else "f32").to(gu.dev())
    pos = two_documents(B, T, cut)
    want = dsc.scan_bwd(**p, act=True, pos=pos)
    fwd = {k: v for k, v in p.items() if k != "dy"}
    y, h, _ = dsc.scan_fwd(**fwd, act=True, pos=pos, final_state=True)
    for name in TOKENS + ("dy",):
        q = dict(p, **{name: p[name].clone()})
        q[name][:, :cut] = bad
        got = dsc.scan_bwd(**q, act=True, pos=pos)
        for k in ("dx", "ddelta", "dz", "dBm", "dCm"):
            assert torch.equal(got[k][:, cut:], want[k][:, cut:]), (name, k)
        q.pop("dy")
        y1, h1, _ = dsc.scan_fwd(**q, act=True, pos=pos, final_state=True)
        assert torch.equal(y1[:, cut:], y[:, cut:]) and torch.equal(h1, h), name
