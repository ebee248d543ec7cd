"""The waits of the differential decode and of the linear attention prompts are
bounded as those of the other decode kernels are: with a variant of the library,
built from a patched copy of the sources, in which one tile is never issued
(and the limit is 2 ms), the launch records PHS_ETIMEOUT and returns, requests
of other CTAs come out as always, and the context stays usable."""
import ctypes
import math
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
    # CTA (0, 0, 0), warp 0 never issues its second chunk
    "phs_diff.cu": [("  auto issue = [&](int c) {  // lane 0\n",
                     "  auto issue = [&](int c) {  // lane 0\n"
                     "    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && "
                     "warp == 0 && c == 1) return;\n")],
    # the first CTA of a launch never issues its second V tile
    "phs_linear.cu": [("          if (!ok) return;\n"
                       "          mbar_arrive_expect_tx(kv_full + 8 * slot, L::kTile);\n",
                       "          if (!ok) return;\n"
                       "          if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && "
                       "tiles == 3) {\n"
                       "            ++tiles;\n"
                       "            return;\n"
                       "          }\n"
                       "          mbar_arrive_expect_tx(kv_full + 8 * slot, L::kTile);\n")],
}
CUDA = ("phs_diff.cu", "phs_linear.cu")


@pytest.fixture(scope="module")
def variant(tmp_path_factory):
    phs_build.build()  # the product objects the variant links against
    d = tmp_path_factory.mktemp("ops_wait_variant")
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
    objs = [str(d / (name[:-3] + ".o")) for name in CUDA]
    procs = [subprocess.Popen([nvcc, *flags, "-c", str(d / name), "-o", o],
                              stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
             for name, o in zip(CUDA, objs)]
    for p in procs:
        out, _ = p.communicate()
        assert p.returncode == 0, out.decode()[-3000:]
    own = [n[:-3] + ".o" for n in CUDA]
    keep = [os.path.join(phs_build.BUILD, n) for n in sorted(os.listdir(phs_build.BUILD))
            if n.endswith(".o") and n not in own]
    so = str(d / "libphs_ops_wait_variant.so")
    subprocess.check_call([nvcc, *phs_build.ARCH, "-shared", "-Xlinker", "-Bsymbolic", "-o",
                           so, *objs, *keep])
    lib = ctypes.CDLL(so)
    for name in ("phs_attn_decode_diff_paged", "phs_diff_workspace_bytes",
                 "phs_linear_attn_prompt", "phs_linear_prompt_workspace_bytes"):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = _lib._SIGS[name]
    return lib


@pytest.mark.parametrize("D,Hq,Hkv,lens", [
    (128, 4, 4, [700, 300]),     # rows alone
    (64, 8, 4, [700, 300]),
    (128, 2, 2, [4000]),         # the sums of segments too
    (64, 2, 2, [4000])])
def test_prompt_wait_runs_out_and_returns(variant, monkeypatch, D, Hq, Hkv, lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    q = synth.normal_bf16((T, Hq, D), 1, device="cuda")
    k = synth.normal_bf16((T, Hkv, D), 2, device="cuda")
    v = synth.normal_bf16((T, Hkv, D), 3, device="cuda")
    decay = torch.full((Hkv,), -0.05, device="cuda")
    args = (q, k, v, dev(cu), max(lens))
    pool = phs.StatePool.zeros(len(lens), Hkv, D)
    ref = phs.linear_attn_prompt(*args, pool, decay)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = phs.StatePool.zeros(len(lens), Hkv, D)
    with monkeypatch.context() as m:
        m.setattr(phs, "lib", lambda: variant)
        out = phs.linear_attn_prompt(*args, bad, decay, out=torch.zeros_like(ref), status=st)
        torch.cuda.synchronize()           # the launches returned
    assert int(st.item()) == -8            # PHS_ETIMEOUT
    if len(lens) > 1:                      # the other heads and requests
        assert torch.equal(out[:, Hq // Hkv:], ref[:, Hq // Hkv:])
        assert torch.equal(bad.s[:, 1:], pool.s[:, 1:])
    again = phs.StatePool.zeros(len(lens), Hkv, D)
    assert torch.equal(phs.linear_attn_prompt(*args, again, decay), ref)
    assert torch.equal(again.s, pool.s)


@pytest.mark.parametrize("D", [64, 128])
def test_diff_wait_runs_out_and_returns(variant, monkeypatch, D):
    B, H, Hv = 3, 4, 2
    lens = np.array([2000, 777, 3001], np.int32)
    bt, npg = synth.block_tables_from_permutation(synth.pages_needed(lens), 5)
    pool = phs.PagedPool(synth.normal_bf16((npg, 2 * Hv, 16, D), 6, device="cuda"),
                         synth.normal_bf16((npg, 2 * Hv, 16, D), 7, device="cuda"))
    q = synth.normal_bf16((B, 2 * H, D), 8, device="cuda")
    vec = torch.full((D,), 0.02, device="cuda")
    w = phs.DiffWeights(vec, vec, vec, vec, 0.5)
    args = (q, pool, dev(bt), dev(lens), int(lens.max()), w)
    ref = phs.attn_decode_diff_paged(*args, out_dtype=torch.float32, tokens_per_split=1024)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(phs, "lib", lambda: variant)
        out = phs.attn_decode_diff_paged(*args, out_dtype=torch.float32, tokens_per_split=1024,
                                         status=st)
        torch.cuda.synchronize()
    assert int(st.item()) == -8
    assert torch.equal(out[1:], ref[1:])
    again = phs.attn_decode_diff_paged(*args, out_dtype=torch.float32, tokens_per_split=1024)
    assert torch.equal(again, ref) and math.isfinite(float(again.sum()))
