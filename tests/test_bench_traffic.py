"""bench.py's key of the captured DRAM traffic: the sources of the kernels that it times."""
import os
import shutil

import bench


def test_the_key_goes_by_the_drafters_sources(tmp_path, monkeypatch):
    name = "speculative_decoding_drafter_hf_gb300"
    src = os.path.join(bench.ROOT, name, "csrc")
    shutil.copytree(src, tmp_path / name / "csrc")
    real = bench.kernel_sources_digest()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_sources_digest() == real

    def touched(f):
        p = tmp_path / name / "csrc" / f
        old = p.read_bytes()
        p.write_bytes(old + b"\n")
        d = bench.kernel_sources_digest()
        p.write_bytes(old)
        return d

    for f in sorted(os.listdir(src)):
        if f.endswith((".cu", ".cuh")):
            assert (touched(f) == real) == (f in bench.TARGET_SIDE), f
    # a new source counts until it is named
    (tmp_path / name / "csrc" / "new.cu").write_text("")
    assert bench.kernel_sources_digest() != real


def test_what_does_not_count_is_no_part_of_what_does():
    """No source that counts includes one that does not."""
    src = os.path.join(bench.ROOT, "speculative_decoding_drafter_hf_gb300", "csrc")
    for f in os.listdir(src):
        if f.endswith((".cu", ".cuh")) and f not in bench.TARGET_SIDE:
            with open(os.path.join(src, f)) as fh:
                text = fh.read()
            assert not any(f'#include "{t}"' in text for t in bench.TARGET_SIDE), f
