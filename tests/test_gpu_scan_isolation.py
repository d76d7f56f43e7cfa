"""Infinite and undefined values stay where the definition has them: documents of
a packed row do not see each other's, also where the time axis is cut between
them, and an infinite value gives the infinite outputs that the formulas give,
for every number of states.  Equal bits, or infinite and undefined outputs in
the same places, are asked for, so no tolerance is needed."""
import numpy as np
import pytest
import torch

import dsc_inputs as di
from tests import gpu_util as gu
from tests import scan_ref as ref
from tests.test_gpu_scan import BF16, F32, dev, f64, make

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


def kinds(a):
    """0 finite, 1 and -1 infinite, 2 undefined."""
    a = a if isinstance(a, np.ndarray) else gu.f64(a)
    return np.where(np.isnan(a), 2, np.where(np.isinf(a), np.sign(a), 0)).astype(int)


def positive(B, T, D, N, dtype, seed, Dk=True, z=False):
    """Inputs whose products keep their sign, rates that decay slowly."""
    p = make(B, T, D, N, 0, 1, dtype, seed, z=z, Dk=Dk)
    for k in ("x", "Bm", "Cm", "Dk", "z"):
        if k in p:
            p[k] = p[k].abs() + 0.5
    p["A"] = -0.01 * (1.0 + torch.arange(N).float()).repeat(D, 1)
    return p


# states that fill no whole number of lanes or waves, and ones that do
STATES = [1, 2, 3, 5, 7, 9, 12, 16, 17, 31, 33, 61]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("B,T", [(2, 40), (1, 400)])
def test_an_infinite_input_gives_infinite_outputs(dsc, B, T, N, dtype):
    """h and y of its channel are infinite from there on, whatever N is; they are
    not undefined, and no other channel sees it."""
    p = positive(B, T, 16, N, dtype, 2400 + N)
    p["x"][0, 21, 3] = float("inf")
    y, h, _ = dsc.scan_fwd(**dev(p), final_state=True)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want, hw, _ = ref.scan_fwd(**f64(p))
    assert (kinds(want)[0, 21:, 3] == 1).all() and np.abs(kinds(want)).sum() == T - 21
    assert np.array_equal(kinds(y), kinds(want)) and np.array_equal(kinds(h), kinds(hw))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
def test_an_infinite_input_of_one_token(dsc, N, dtype):
    B, D = 2, 72
    p = positive(B, 1, D, N, dtype, 2500 + N)
    p["x"][0, 0, 3] = float("inf")
    with np.errstate(all="ignore"):
        want, hw, _ = ref.scan_fwd(**f64(p))
    tok = {k: v[:, 0] if v.dim() >= 3 else v for k, v in dev(p).items()}
    h = torch.zeros(B, D, N, device=gu.dev())
    y = dsc.scan_decode(**tok, h=h)
    torch.cuda.synchronize()
    assert np.array_equal(kinds(y), kinds(want[:, 0])) and np.array_equal(kinds(h), kinds(hw))
    assert kinds(want)[0, 0, 3] == 1


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", STATES)
@pytest.mark.parametrize("B,T", [(2, 40), (1, 400)])
def test_an_infinite_gradient(dsc, B, T, N, dtype):
    """dx of its channel is infinite up to there, dBm in every state, dCm at its
    token; ddelta, a difference of infinities, is undefined where the formula is."""
    p = positive(B, T, 16, N, dtype, 2600 + N)
    dy = di.randn((B, T, 16), 1.0, 2700, "bf16" if dtype == BF16 else "f32")
    dy[0, 21, 3] = float("inf")
    g = dsc.scan_bwd(**dev(p), dy=dy.to(gu.dev()))
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want = ref.scan_bwd(**f64(p), dy=gu.f64(dy))
    assert (kinds(want["dx"])[0, :22, 3] == 1).all() and np.abs(kinds(want["dx"])).sum() == 22
    for k in ("dx", "ddelta", "dBm", "dCm"):
        assert np.array_equal(kinds(g[k]), kinds(want[k])), k


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("N", [5, 16])
def test_an_absent_Dk_adds_nothing(dsc, N, z, dtype):
    """Without Dk, an infinite u or dp meets no zero in its place."""
    B, T, D = 1, 40, 16
    p = positive(B, T, D, N, dtype, 2800 + N, Dk=False, z=z)
    p["x"][0, 21, 3] = float("inf")
    q = f64(p)
    with np.errstate(all="ignore"):
        want, hw, _ = ref.scan_fwd(**q)
    assert (kinds(want)[0, 21:, 3] == 1).all()
    y, h, _ = dsc.scan_fwd(**dev(p), final_state=True)
    assert np.array_equal(kinds(y), kinds(want)) and np.array_equal(kinds(h), kinds(hw))
    seq = {k: v for k, v in dev(p).items() if v.dim() >= 3}
    tok = {k: v[:, 21] for k, v in seq.items()}
    hd = torch.zeros(B, D, N, device=gu.dev())
    y = dsc.scan_decode(**dict(dev(p), **tok), h=hd)
    assert kinds(y)[0, 3] == 1 and np.abs(kinds(y)).sum() == 1
    dy = di.randn((B, T, D), 1.0, 2900, "bf16" if dtype == BF16 else "f32")
    g = dsc.scan_bwd(**dev(p), dy=dy.to(gu.dev()))
    with np.errstate(all="ignore"):
        want = ref.scan_bwd(**q, dy=gu.f64(dy))
    if z:
        assert np.array_equal(kinds(g["dz"]), kinds(want["dz"]))
        assert (np.abs(kinds(want["dz"])[0, 21:, 3]) == 1).all()
    # an infinite gradient
    p = positive(B, T, D, N, dtype, 2850 + N, Dk=False, z=z)
    dy[0, 21, 3] = float("inf")
    g = dsc.scan_bwd(**dev(p), dy=dy.to(gu.dev()))
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want = ref.scan_bwd(**f64(p), dy=gu.f64(dy))
    assert np.array_equal(kinds(g["dx"]), kinds(want["dx"]))
    assert (kinds(want["dx"])[0, :22, 3] == 1).all()
