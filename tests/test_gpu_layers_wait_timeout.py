"""The waits of the selective scan's prompts are bounded as those of the other
kernels are: with a variant of the library, built from a patched copy of the
sources, in which one tile is never issued (and the limit is 2 ms), the launch
records PHS_ETIMEOUT and returns, requests and heads of other CTAs come out as
always, and the context stays usable."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import paged_hybrid_sliding_gb300 as phs
import synth
from paged_hybrid_sliding_gb300 import _lib
from paged_hybrid_sliding_gb300 import build as phs_build
from gpu_util import dev

pytestmark = pytest.mark.gpu

PATCHES = {
    "phs_common.cuh": [("constexpr uint64_t kWaitLimitNs = 1000000000ull;",
                        "constexpr uint64_t kWaitLimitNs = 2000000ull;")],
    # the first CTA of a launch never issues its second chunk's last tile
    "phs_scan_prompt.cu": [("          if (!ok) return;\n"
                            "          mbar_arrive_expect_tx(full_of(tiles), halves * kHalf);\n",
                            "          if (!ok) return;\n"
                            "          if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && "
                            "tiles == 2 * L::kPer - 1) {\n"
                            "            ++tiles;\n"
                            "            return;\n"
                            "          }\n"
                            "          mbar_arrive_expect_tx(full_of(tiles), halves * kHalf);\n")],
}


@pytest.fixture(scope="module")
def variant(tmp_path_factory):
    phs_build.build()  # the product objects the variant links against
    d = tmp_path_factory.mktemp("layers_wait_variant")
    src = os.path.join(phs_build.HERE, "csrc")
    for name in os.listdir(src):
        shutil.copy(os.path.join(src, name), d / name)
    for name, changes in PATCHES.items():
        text = (d / name).read_text()
        for old, new in changes:
            assert text.count(old) == 1, (name, old)
            text = text.replace(old, new)
        (d / name).write_text(text)
    nvcc = phs_build.nvcc_path()
    flags = [f if f != phs_build.CSRC else str(d) for f in phs_build._flags()]
    obj = str(d / "phs_scan_prompt.o")
    subprocess.check_call([nvcc, *flags, "-c", str(d / "phs_scan_prompt.cu"), "-o", obj])
    keep = [os.path.join(phs_build.BUILD, n) for n in sorted(os.listdir(phs_build.BUILD))
            if n.endswith(".o") and n != "phs_scan_prompt.o"]
    so = str(d / "libphs_layers_wait_variant.so")
    subprocess.check_call([nvcc, *phs_build.ARCH, "-shared", "-Xlinker", "-Bsymbolic", "-o", so, obj,
                           *keep])
    lib = ctypes.CDLL(so)
    for name in ("phs_selective_scan_prompt", "phs_scan_prompt_workspace_bytes"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = _lib._SIGS[name]
    return lib


@pytest.mark.parametrize("H,G,P,N,lens", [
    (4, 1, 64, 128, [700, 300]),    # rows alone
    (6, 2, 64, 64, [700, 300]),
    (2, 1, 128, 128, [700, 300]),
    (2, 1, 64, 128, [4000]),        # the sums of segments too
    (1, 1, 64, 64, [4000])])
def test_prompt_wait_runs_out_and_returns(variant, monkeypatch, H, G, P, N, lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, B = int(cu[-1]), len(lens)
    x, dt = synth.normal_bf16((T, H, P), 1, device="cuda"), synth.normal_bf16((T, H), 2, device="cuda")
    b, c = (synth.normal_bf16((T, G, N), s, device="cuda") for s in (3, 4))
    w = phs.ScanWeights(torch.full((H,), -0.5, device="cuda"))
    args = (x, dt, b, c, dev(cu), max(lens))
    pool = phs.ScanPool.zeros(B, H, P, N)
    want = phs.selective_scan_prompt(*args, pool, w)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = phs.ScanPool.zeros(B, H, P, N)
    with monkeypatch.context() as m:
        m.setattr(phs, "lib", lambda: variant)
        out = phs.selective_scan_prompt(*args, bad, w, out=torch.zeros_like(want), status=st)
        torch.cuda.synchronize()           # the launches returned
    assert int(st.item()) == -8            # PHS_ETIMEOUT
    if B > 1:                              # the other heads and requests
        first = 1 if P == 128 or H // G % 2 else 2
        assert torch.equal(out[:, first:], want[:, first:])
        assert torch.equal(bad.s[:, first:], pool.s[:, first:])
        # (the longest request has the first CTA where there are more CTAs than SMs)
        assert torch.equal(out[700:], want[700:]) and torch.equal(bad.s[1], pool.s[1])
    again = phs.ScanPool.zeros(B, H, P, N)
    assert torch.equal(phs.selective_scan_prompt(*args, again, w), want)
    assert torch.equal(again.s, pool.s)
