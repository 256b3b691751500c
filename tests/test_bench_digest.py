"""The DRAM figures that bench.py takes from committed captures are dropped once a source they depend on changes."""
import os
import shutil

import bench

CSRC = os.path.join("multiresolution_hash_grid_b200", "csrc")


def test_digest_covers_what_chooses_and_launches_the_captured_kernels(tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    whole = bench.csrc_digest()
    for name in sorted(os.listdir(tmp_path / CSRC)):
        with open(tmp_path / CSRC / name) as f:
            text = f.read()
        with open(tmp_path / CSRC / name, "w") as f:
            f.write(text + "\n")
        # the layers' and the optimiser's kernels are not among the captured ones
        assert (bench.csrc_digest() == whole) == (name in ("hg_linear.cuh", "hg_adamw.cuh")), name
        with open(tmp_path / CSRC / name, "w") as f:
            f.write(text)
    assert bench.csrc_digest() == whole
