"""The build's own checks: the scan backward's units with the fullest registers
compile without a spill, a spill is refused, and a build that fails leaves no
library behind that would pass for its result."""
import os

import pytest

import __graft_entry__ as ge


@pytest.fixture()
def builder(tmp_path, monkeypatch):
    b = ge._library_builder()
    monkeypatch.setattr(b, "OBJ", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    return b


@pytest.mark.parametrize("source", ["scan_bwd_f32.hip", "scan_bwd_bf16.hip"])
def test_the_scan_backward_does_not_spill(builder, source):
    """Four waves a workgroup: two workgroups a CU leave a wave 256 registers."""
    unit = (source, ("-DDSC_SCAN_NW=4",))
    assert unit in builder.SOURCES
    _, _, remarks = builder._compile(unit)
    rows = builder._resources(remarks)
    main = [r for r in rows if "scan_bwd_kernel" in r["name"]]
    assert len(main) == 8
    assert {r["name"]: r["ScratchSize [bytes/lane]"] for r in rows} == \
        {r["name"]: "0" for r in rows}


def test_a_spill_is_refused(builder):
    row = {"name": "_ZN3dsc11some_kernelIfEEv", "ScratchSize [bytes/lane]": "60"}
    with pytest.raises(RuntimeError, match="spill"):
        builder._refuse_spills([dict(row, **{"ScratchSize [bytes/lane]": "0"}), row])
    builder._refuse_spills([dict(row, **{"ScratchSize [bytes/lane]": "0"})])


def test_a_failed_build_leaves_no_library(builder, monkeypatch):
    with open(builder.LIB, "w") as f:
        f.write("an older build's")
    monkeypatch.setattr(builder, "SOURCES", [("no_such_source.hip", ())])
    with pytest.raises(RuntimeError):
        builder.build(jobs=1)
    assert not os.path.exists(builder.LIB)


def test_the_scan_dispatch_holds_no_kernels_of_the_units(builder):
    """scan_bwd.hip compiles its own kernel; the others come from the units that
    are compiled once per number of waves, and once only."""
    _, _, remarks = builder._compile(("scan_bwd.hip", ()))
    names = [r["name"] for r in builder._resources(remarks)]
    assert len(names) == 2 and all("scan_bwd_finish_kernel" in n for n in names), names
