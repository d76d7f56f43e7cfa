"""The scan's tilings as scan_launch.hpp chooses them: a host program prints the
plans of a list of shapes."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include <stdio.h>
#include "scan_launch.hpp"
int main() {
  long long B, T, D;
  int G, N, W, bf16;
  while (scanf("%lld %lld %lld %d %d %d %d", &B, &T, &D, &G, &N, &W, &bf16) == 7) {
    const dsc::ScanPlan f = dsc::scan_plan(B, T, D, G, N);
    const dsc::ScanBwdPlan q = dsc::scan_bwd_plan(B, T, D, G, N, W, bf16 != 0);
    printf("%d %d %d %d %lld %zu %d %d %d %d %lld %zu %d %d %d\\n", f.ns, f.nw, f.nc, f.tc,
           (long long)f.cols, f.total, q.ns, q.nw, q.nc, q.tc, (long long)q.cols, q.total, q.tiles,
           dsc::scan_bwd_tile(q.ns, q.nw), dsc::scan_bwd_resident(bf16 != 0, q.nw, W));
  }
}
"""
FWD, BWD = ("ns", "nw", "nc", "tc", "cols", "total"), ("ns", "nw", "nc", "tc", "cols", "total",
                                                       "tiles", "tile", "resident")


def build(folder):
    src, exe = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "dynamic_short_causal_amd", "csrc"), src, "-o", exe],
                   check=True)
    return exe


def plans(exe, shapes):
    """(forward, backward) dicts of (B, T, D, G, N, W, bf16) shapes."""
    text = "\n".join(" ".join(str(int(v)) for v in s) for s in shapes)
    out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
    rows = [[int(v) for v in line.split()] for line in out.splitlines()]
    assert len(rows) == len(shapes)
    return [(dict(zip(FWD, r)), dict(zip(BWD, r[len(FWD):]))) for r in rows]
