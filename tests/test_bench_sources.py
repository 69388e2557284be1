"""The recorded DRAM traffic of a step is tied to every source that a step is made from."""
import json
import os

import bench

CSRC = os.path.join(bench.ROOT, "decode_megakernel_interpreter_b200", "csrc")


def test_every_source_but_the_serving_operators_counts():
    assert set(bench.SERVING) <= set(os.listdir(CSRC))
    assert set(bench.step_sources()) == set(os.listdir(CSRC)) - set(bench.SERVING)
    assert {"api.cu", "noalloc.cu", "interp_body.cuh", "planner.cpp", "mk_internal.h"} <= set(bench.step_sources())
    assert not any(f.startswith("interp") for f in bench.SERVING)


def test_a_change_of_any_of_them_shows(tmp_path, monkeypatch):
    d = tmp_path / "decode_megakernel_interpreter_b200" / "csrc"
    d.mkdir(parents=True)
    for f in os.listdir(CSRC):
        (d / f).write_bytes(open(os.path.join(CSRC, f), "rb").read())
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    was = bench.src_hash()
    for f in bench.step_sources():
        before = (d / f).read_bytes()
        (d / f).write_bytes(before + b" ")
        assert bench.src_hash() != was, f
        (d / f).write_bytes(before)
    for f in bench.SERVING:
        (d / f).write_bytes(b"")
    assert bench.src_hash() == was


def test_the_record_names_its_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        for e in json.load(f).values():
            assert len(e["src_hash"]) == 16 and e["dram_bytes_per_launch"] > 0
