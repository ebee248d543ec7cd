"""The device headers go together: one source may include them all."""
import glob
import os
import subprocess

import pytest

from paged_hybrid_sliding_gb300 import build as phs_build


def test_one_source_may_include_every_header(tmp_path):
    try:
        nvcc = phs_build.nvcc_path()
    except RuntimeError:
        pytest.skip("no nvcc")
    names = sorted(os.path.basename(p) for p in glob.glob(os.path.join(phs_build.CSRC, "*.cuh")) +
                   glob.glob(os.path.join(phs_build.CSRC, "*.h")))
    src = tmp_path / "all.cu"
    src.write_text("".join(f'#include "{n}"\n' for n in names))
    r = subprocess.run([nvcc, *phs_build._flags(), "-c", str(src), "-o", str(tmp_path / "all.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
