"""The scan's tilings: they cover the time axis, the number of chunks is the one
that its rule prefers once rounded to whole tiles, and the GPU tests of single
tilings have sizes that reach them."""
import math
import random

import pytest
import torch

from tests import scan_plan
from tests import test_gpu_scan_chunks as chunks

CUS = 256


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = scan_plan.build(str(tmp_path_factory.mktemp("plan")))
    return lambda shapes: scan_plan.plans(exe, shapes)


def drawn(n):
    r = random.Random(7)
    out = []
    for _ in range(n):
        G = r.choice([1, 1, 2, 8])
        out.append((int(2 ** r.uniform(0, 8)), int(2 ** r.uniform(0, 16)),
                    8 * G * int(2 ** r.uniform(0, 9)), G, r.randint(1, 64), r.randint(0, 8),
                    r.randint(0, 1)))
    return out


def test_chunks_cover_the_axis(plans):
    shapes = drawn(2000)
    for s, both in zip(shapes, plans(shapes)):
        for p in both:
            assert p["nc"] >= 1 and (p["nc"] - 1) * p["tc"] < s[1] <= p["nc"] * p["tc"], s
            assert p["ns"] * p["nw"] >= s[4], s


def test_rounding_keeps_the_backwards_choice(plans):
    """Rounds of workgroups times the length of a chunk is what a count of chunks
    is chosen by: none that its whole tiles allow is better by a tenth, whole rows
    among them, where a call is more than a few tiles long."""
    shapes = [s for s in drawn(2000) if s[1] >= 512]
    shapes += [(8, 2048, 1088, 1, 16, 4, 1), (9, 2048, 1024, 1, 16, 4, 1),
               (6, 2048, 1408, 1, 16, 4, 1), (5, 2048, 1088, 1, 64, 4, 1)]
    for s, (_, p) in zip(shapes, plans(shapes)):
        slots, tiles = CUS * p["resident"], p["tiles"]

        def work(n_chunks, length):
            extra = 0 if n_chunks == 1 else 1 + n_chunks / 20
            return math.ceil(p["cols"] * n_chunks / slots) * (length + extra)
        mine = work(p["nc"], p["tc"] // p["tile"])
        for k in range(1, min(64, tiles) + 1):
            length = math.ceil(tiles / k)
            n = math.ceil(tiles / length)
            assert mine <= 1.1 * work(n, length), (s, p["nc"], n)


def test_residents_are_those_of_the_types(plans):
    got = [p["resident"] for _, p in plans([(8, 512, 512, 1, 16, W, b) for W in (4, 8)
                                            for b in (0, 1)])]
    assert got == [2, 2, 1, 2]        # fp32 with eight taps has one workgroup a CU


def shape(c):
    return c.B, c.T, c.D, c.G, c.N, c.W, c.dtype == torch.bfloat16


def test_the_gpu_tests_reach_their_tilings(plans):
    for c, (f, _) in zip(chunks.FORWARD, plans([shape(c) for c in chunks.FORWARD])):
        assert (f["nc"], f["ns"]) == (c.chunks, c.states), (c, f)
    for c, (_, b) in zip(chunks.BACKWARD, plans([shape(c) for c in chunks.BACKWARD])):
        assert (b["nc"], b["nw"]) == (c.chunks, c.waves), (c, b)
    assert {c.chunks for c in chunks.BACKWARD} >= {1, 2, 8}
