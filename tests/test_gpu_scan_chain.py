"""The scan behind this library's dynamic convolution (no convolution of its own),
on whole and on packed rows.

Tolerance: the convolution's fp32 outputs are within 1e-5 of the oracle's
(gpu_util.py); the scan adds them up over T tokens with steps below one and B and
C of order one, so its outputs differ by at most 1e-5 times the sum over a
decaying history of dt |B| |C| N, some tens here; 1e-3 of the largest output, which
is of order one, leaves room, and a tap or a channel out of place shows at 0.1.
"""
import numpy as np
import pytest
import torch

import dsc_inputs as di
from tests import gpu_util as gu
from tests import scan_ref as ref
from tests.test_gpu_scan import F32, dev, documents, f64, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("form", ["headwise", "lowrank"])
def test_dynamic_convolution_into_the_scan(orc, form, packed):
    import dynamic_short_causal_amd as dsc
    B, T, D, N, W, H = 2, 90, 64, 16, 4, 8
    p = make(B, T, D, N, 0, 1, F32, 3500)
    pos = documents(B, T, 3501)
    x = p["x"]
    X, P = gu.f64(x), pos.numpy()
    if form == "headwise":
        w = di.randn((B, T, D // H, W), 0.5, 3502, "f32")
        args, exact = (x, w), (X, gu.f64(w))
        tail = (H, False, True)
    else:
        z, U = di.randn((B, T, 16), 1.0, 3503, "f32"), di.randn((16, D * W), 0.125, 3504, "f32")
        args, exact = (x, z, U), (X, gu.f64(z), gu.f64(U))
        tail = (W, 1, False, True)
    if packed:
        u = getattr(dsc, form + "_fwd_varlen")(*[t.to(gu.dev()) for t in args],
                                               pos.to(gu.dev()), *tail)
        s = getattr(orc, form + "_fwd_vl")(*exact, P, *(tail[:1] if form == "headwise" else
                                                        tail[:2]), act=True)
    else:
        u = getattr(dsc, form + "_fwd")(*[t.to(gu.dev()) for t in args], *tail)
        s = getattr(orc, form + "_fwd")(*exact, *(tail[:1] if form == "headwise" else tail[:2]),
                                        act=True)
    more = dict(pos=pos) if packed else {}
    q = dev(dict(p, **more))
    q["x"] = u
    y, h, conv = dsc.scan_fwd(**q, final_state=True)
    torch.cuda.synchronize()
    e = f64(dict(p, **more))
    e["x"] = s
    want, hw, _ = ref.scan_fwd(**e)
    assert conv.shape == (B, 0, D)
    for name, got, exact_ in (("y", y, want), ("h", h, hw)):
        a, m = gu.err(got, exact_)
        gu.say(f"    {name}: {a:.2e} of {m:.2e}")
        assert a <= 1e-3 * m
    # one token further by both one-token forms, on whole rows
    if not packed and form == "headwise":
        st = dsc.decode_state(x.to(gu.dev()), W)
        x1, w1 = di.randn((B, D), 1.0, 3510, "f32"), di.randn((B, D // H, W), 0.5, 3511, "f32")
        u1 = dsc.headwise_decode(x1.to(gu.dev()), w1.to(gu.dev()), st, H, act=True)
        t = make(B, 1, D, N, 0, 1, F32, 3512)
        y1 = dsc.scan_decode(u1, t["delta"][:, 0].to(gu.dev()), q["A"],
                             *(t[k][:, 0].to(gu.dev()) for k in ("Bm", "Cm")), h=h, Dk=q["Dk"],
                             z=t["z"][:, 0].to(gu.dev()), dt_bias=q["dt_bias"])
        torch.cuda.synchronize()
        s_all = orc.headwise_fwd(np.concatenate([X, gu.f64(x1)[:, None]], 1),
                                 np.concatenate([gu.f64(w), gu.f64(w1)[:, None]], 1), H, act=True)
        g = dict(f64(t), x=s_all[:, -1:], A=e["A"], Dk=e["Dk"], dt_bias=e["dt_bias"])
        want1, _, _ = ref.scan_fwd(**g, h0=hw)
        a, m = gu.err(y1, want1[:, 0])
        assert a <= 1e-3 * m
