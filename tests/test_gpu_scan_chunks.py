"""The scan where its time axis is cut, and where it is not, at sizes that are
known to take each tiling (test_scan_plan.py asks the plans): forward calls in
chunks for every number of state groups, several sequences and groups of B and C,
backward calls whole, in two, four and eight chunks.  Tolerances as in
test_gpu_scan.py."""
import collections

import pytest

import dsc_inputs as di
from tests.test_gpu_scan import BF16, F32, documents, make, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

Fwd = collections.namedtuple("Fwd", "B T D G N W dtype packed chunks states")
Bwd = collections.namedtuple("Bwd", "B T D G N W dtype packed chunks waves")

FORWARD = [Fwd(2, 581, 144, 2, N, W, dtype, packed, 10, 4)
           for N, W, dtype, packed in [
               (3, 4, BF16, True), (4, 4, F32, False), (4, 8, BF16, True), (8, 3, BF16, False),
               (7, 8, F32, True), (16, 8, F32, True), (16, 2, BF16, False), (13, 4, F32, True),
               (24, 4, BF16, True), (24, 8, F32, False), (33, 4, BF16, False), (64, 8, BF16, True),
               (64, 4, F32, True)]]
BACKWARD = [
    Bwd(3, 510, 512, 64, 16, 4, BF16, False, 8, 4), Bwd(3, 509, 512, 64, 12, 4, F32, True, 8, 4),
    Bwd(3, 510, 512, 64, 16, 8, F32, False, 4, 4), Bwd(6, 254, 512, 64, 6, 8, BF16, True, 8, 2),
    Bwd(6, 254, 512, 64, 6, 8, F32, False, 4, 2), Bwd(3, 250, 256, 32, 40, 3, F32, True, 8, 8),
    Bwd(6, 255, 512, 64, 3, 4, F32, False, 8, 1), Bwd(3, 505, 256, 32, 24, 4, BF16, True, 8, 8),
    Bwd(8, 70, 512, 64, 16, 4, BF16, True, 1, 4), Bwd(8, 70, 512, 64, 12, 8, F32, False, 1, 4),
    Bwd(16, 50, 512, 64, 6, 4, BF16, False, 1, 2), Bwd(4, 60, 512, 64, 40, 4, F32, True, 1, 8),
    Bwd(16, 50, 512, 64, 4, 4, F32, True, 1, 1), Bwd(60, 67, 512, 1, 6, 8, BF16, True, 2, 2)]


def name(c):
    return "-".join(str(v).replace("torch.", "") for v in c)


@pytest.mark.parametrize("c", FORWARD, ids=name)
def test_cut_forward(c):
    import dynamic_short_causal_amd as dsc
    p = make(c.B, c.T, c.D, c.N, c.W, c.G, c.dtype, 3000 + c.N)
    if not c.packed:
        run_fwd(dsc, p, c.W)
    more = dict(h0=di.randn((c.B, c.D, c.N), 1.0, 3100, "f32"),
                conv0=di.randn((c.B, c.W - 1, c.D), 1.0, 3101,
                               "bf16" if c.dtype == BF16 else "f32"))
    if c.packed:
        more["pos"] = documents(c.B, c.T, 3102 + c.N, start=False)
    run_fwd(dsc, p, c.W, residual=c.packed, **more)


@pytest.mark.parametrize("c", BACKWARD, ids=name)
def test_chunks_of_the_backward(c):
    import dynamic_short_causal_amd as dsc
    p = make(c.B, c.T, c.D, c.N, c.W, c.G, c.dtype, 3200 + c.N)
    run_bwd(dsc, p, pos=documents(c.B, c.T, 3300 + c.N) if c.packed else None)
