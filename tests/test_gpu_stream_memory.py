"""Calls queued on a stream that is not the current one: their workspaces and
outputs are not handed to the current stream's next tensors while the kernels
still use them."""
import pytest
import torch

import dsc_inputs as di
from tests.test_gpu_scan import BF16, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsc():
    import dynamic_short_causal_amd as d
    return d


def calls(dsc):
    def c(t):
        return t.cuda()
    B, T, D, W = 2, 300, 1024, 4
    x, dy = (c(di.randn((B, T, D), 1.0, 30 + i, "bf16")) for i in range(2))
    w = c(di.randn((B, T, 64, W), 0.5, 32, "bf16"))
    z = c(di.randn((B, T, 16), 1.0, 33, "bf16"))
    U = c(di.randn((16, D * W), 0.125, 34, "bf16"))
    ws = c(di.randn((D, W), 0.5, 35, "bf16"))
    pos = torch.arange(T, dtype=torch.int32).repeat(B, 1).cuda()
    p = {k: c(v) for k, v in make(1, 1100, 64, 16, W, 1, BF16, 36).items()}  # cut both ways
    rows = x.view(-1, D)
    _, mean, rstd = dsc.layernorm_fwd(rows, ws[:, 0].contiguous())
    return {
        "headwise_fwd": lambda s: dsc.headwise_fwd(x, w, 16, stream=s),
        "headwise_bwd": lambda s: dsc.headwise_bwd(x, w, dy, 16, False, False, s),
        "lowrank_fwd": lambda s: dsc.lowrank_fwd(x, z, U, W, 1, stream=s),
        "lowrank_bwd": lambda s: dsc.lowrank_bwd(x, z, U, dy, W, 1, stream=s),
        "lowrank_bwd_varlen": lambda s: dsc.lowrank_bwd_varlen(x, z, U, pos, dy, W, 1, stream=s),
        "static_bwd": lambda s: dsc.static_bwd(x, ws, dy, 1, stream=s),
        "decode_state": lambda s: dsc.decode_state(x, W, s),
        "scan_fwd": lambda s: dsc.scan_fwd(**p, act=True, final_state=True, stream=s),
        "scan_bwd": lambda s: dsc.scan_bwd(**p, dy=p["z"], act=True, stream=s),
        "layernorm_fwd": lambda s: dsc.layernorm_fwd(rows, stream=s),
        "layernorm_bwd": lambda s: dsc.layernorm_bwd(rows, None, dy.view(-1, D), mean, rstd,
                                                     stream=s),
    }


NAMES = ["headwise_fwd", "headwise_bwd", "lowrank_fwd", "lowrank_bwd", "lowrank_bwd_varlen",
         "static_bwd", "decode_state", "scan_fwd", "scan_bwd", "layernorm_fwd", "layernorm_bwd"]


def tensors(out):
    return list(out.values()) if isinstance(out, dict) else \
        list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("keep", [True, False], ids=["outputs kept", "outputs dropped"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_another_stream(dsc, name, keep):
    call = calls(dsc)[name]
    want = [t.clone() for t in tensors(call(None))]
    big = torch.randn(4096, 4096, device="cuda", dtype=BF16)
    prod = torch.empty_like(big)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(60):           # some milliseconds: the call's kernels start after what
            torch.mm(big, big, out=prod)  # follows on the current stream
    out = call(s)
    if not keep:
        out = None
    # the current stream's next tensors, of every size that the call may have released
    sizes = [t.numel() * t.element_size() for t in want] + [1 << k for k in range(9, 26)]
    mine = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in sizes for _ in (0, 1)]
    torch.cuda.synchronize()
    for t in mine:
        assert int(t.min()) == int(t.max()) == 0x5a, t.numel()
    if keep:
        for a, b in zip(tensors(out), want):
            assert torch.equal(a, b)


def test_the_current_stream_given_by_name_is_as_none_given(dsc):
    call = calls(dsc)["scan_fwd"]
    want = call(None)
    got = call(torch.cuda.current_stream())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
