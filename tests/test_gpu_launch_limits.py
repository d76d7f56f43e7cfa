"""Calls whose workgroups have 2^32 threads or more together, which one launch
does not run: their last rows, sequences and columns against the 64-bit
reference.  Tolerances as in test_gpu_scan.py and test_gpu_norm.py."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from tests import scan_ref as ref
from tests.test_gpu_scan import BF16, EPS, F32, close, f64

pytestmark = pytest.mark.gpu

MANY = (1 << 26) + 5    # times 64 lanes: more than 2^32


@pytest.fixture(scope="module")
def dsc():
    import dynamic_short_causal_amd as d
    yield d
    torch.cuda.empty_cache()


def normal(*shape, dtype=BF16, seed=1):
    g = torch.Generator(device=gu.dev()).manual_seed(seed)
    return torch.empty(*shape, dtype=dtype, device=gu.dev()).normal_(generator=g)


def inputs(B, T, N):
    p = {k: normal(B, T, 8, seed=i) for i, k in enumerate(("x", "delta"))}
    p.update({k: normal(B, T, 1, N, seed=9 + i) for i, k in enumerate(("Bm", "Cm"))})
    p["A"] = -torch.arange(1.0, N + 1, device=gu.dev()).repeat(8, 1)
    return p


def ends(p, n=3):
    """The last n sequences and the first one, on the host."""
    return {k: v.cpu() if k == "A" else torch.cat([v[:1], v[-n:]]).cpu() for k, v in p.items()}


def test_many_rows_of_layer_norm(dsc):
    x = normal(MANY, 8)
    y, m, r = dsc.layernorm_fwd(x)
    rows = torch.cat([x[:2], x[-3:]]).cpu()
    want, mean, rstd = ref.layernorm_fwd(gu.f64(rows), None, None, 1e-5)

    def both(t):
        return torch.cat([t[:2], t[-3:]])
    big, spread = float(np.abs(gu.f64(rows)).max()), float((1.0 / rstd).min())
    rel = 4 * EPS * np.sqrt(8) * (1.0 + big / spread) + 8 * EPS
    for got, exact, lim in ((y, want, 2 * rel + 2.0 ** -8), (m, mean, rel), (r, rstd, rel)):
        a, top = gu.err(both(got), exact)
        assert a <= lim * max(top, 1.0), (a, top)


def test_a_very_long_row_of_layer_norm_backward(dsc):
    """16 D threads add dw and db: the last columns of 2^28 and some."""
    D = (1 << 28) + 64
    x, dy = normal(1, D), normal(1, D, seed=2)
    mean = torch.zeros(1, device=gu.dev())
    rstd = torch.ones(1, device=gu.dev())
    _, dw, db = dsc.layernorm_bwd(x, None, dy, mean, rstd)
    for part in (slice(0, 9), slice(D - 9, D)):
        w = gu.f64(x[0, part]) * gu.f64(dy[0, part])
        assert np.abs(gu.f64(dw[part]) - w).max() <= 2.0 ** -8 * np.abs(w).max()
        assert np.array_equal(gu.f64(db[part]), gu.f64(dy[0, part]))


def test_many_sequences_forward(dsc):
    p = inputs(MANY, 1, 1)
    y, h, _ = dsc.scan_fwd(**p, final_state=True)
    want, hw, _ = ref.scan_fwd(**f64(ends(p)))
    close("y", torch.cat([y[:1], y[-3:]]), want, BF16, 2, 1.0)
    close("h", torch.cat([h[:1], h[-3:]]), hw, F32, 2, 1.0)


def test_many_sequences_of_one_token(dsc):
    p = inputs(MANY, 1, 1)
    tok = {k: v if k == "A" else v[:, 0] for k, v in p.items()}
    h = torch.zeros(MANY, 8, 1, device=gu.dev())
    y = dsc.scan_decode(**tok, h=h)
    want, hw, _ = ref.scan_fwd(**f64(ends(p)))
    close("y", torch.cat([y[:1], y[-3:]]), want[:, 0], BF16, 2, 1.0)
    close("h", torch.cat([h[:1], h[-3:]]), hw, F32, 2, 1.0)


def backward(dsc, B, T, N):
    p = inputs(B, T, N)
    dy = normal(B, T, 8, seed=20)
    g = dsc.scan_bwd(**p, dy=dy)
    want = ref.scan_bwd(**f64(ends(p)), dy=gu.f64(torch.cat([dy[:1], dy[-3:]])))
    for k in ("dx", "ddelta", "dBm", "dCm"):
        got = torch.cat([g[k][:1], g[k][-3:]])
        close(k, got, want[k], BF16, T + N + 8, 1.0)


def test_many_sequences_backward(dsc):
    backward(dsc, MANY, 1, 1)


def test_many_gradients_of_B_and_C(dsc):
    """The last launch has a thread for each element of dBm and dCm."""
    backward(dsc, (1 << 19) + 3, 64, 64)


@pytest.mark.parametrize("name", ["headwise_fwd", "headwise_bwd", "static_fwd", "lowrank_fwd",
                                  "lowrank_bwd", "decode_state"])
def test_the_convolutions_refuse_what_one_launch_does_not_run(dsc, name):
    """One workgroup a sequence of one token: they are not cut into launches, and
    leave nothing unwritten without saying so."""
    B, D = (1 << 24) + 1, 8
    if name == "decode_state":
        B = (1 << 32) // 7 + 1
        x = torch.empty(B, 1, D, dtype=BF16, device=gu.dev())
        with pytest.raises(dsc.DscError):
            dsc.decode_state(x, 8)
        return
    x = torch.zeros(B, 1, D, dtype=BF16, device=gu.dev())
    w = torch.zeros(B, 1, 1, 4, dtype=BF16, device=gu.dev())
    z = torch.zeros(B, 1, 4, dtype=BF16, device=gu.dev())
    U = torch.zeros(4, D * 4, dtype=BF16, device=gu.dev())
    call = {"headwise_fwd": lambda: dsc.headwise_fwd(x, w, 8),
            "headwise_bwd": lambda: dsc.headwise_bwd(x, w, x, 8),
            "static_fwd": lambda: dsc.static_fwd(x, U.view(4 * D, 4)[:D].contiguous(), 1),
            "lowrank_fwd": lambda: dsc.lowrank_fwd(x, z, U, 4, 1),
            "lowrank_bwd": lambda: dsc.lowrank_bwd(x, z, U, x, 4, 1)}[name]
    with pytest.raises(dsc.DscError):
        call()
