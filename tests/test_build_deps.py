"""CPU test of the build's staleness check: every source and header that the library is made of is watched."""
import glob
import os

from gated_delta_rule_40_gb300 import build


def test_every_source_and_header_is_watched():
    files = [f for d in (build.CSRC, os.path.join(build.ROOT, "include")) for f in glob.glob(os.path.join(d, "*"))]
    assert any(f.endswith(".h") for f in files if os.path.dirname(f) == build.CSRC)
    missing = {os.path.abspath(f) for f in files} - {os.path.abspath(f) for f in build._deps()}
    assert not missing, sorted(missing)


def test_an_edited_header_makes_the_library_stale(tmp_path, monkeypatch):
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("a.cu", "a.cuh", "a.h"):
        (csrc / name).write_text("")
        os.utime(csrc / name, (1000, 1000))
    lib = tmp_path / "lib.so"
    lib.write_text("")
    monkeypatch.setattr(build, "CSRC", str(csrc))
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "__file__", str(csrc / "a.cu"))
    os.utime(lib, (2000, 2000))
    assert build.up_to_date()
    for name in ("a.cu", "a.cuh", "a.h"):
        os.utime(csrc / name, (3000, 3000))
        assert not build.up_to_date(), name
        os.utime(csrc / name, (1000, 1000))
