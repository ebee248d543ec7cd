"""Prompts of the selective scan where they can go wrong unseen: workspaces past
32-bit counts, weights of single tokens, the order in which a call's requests
are taken, what a state keeps of its tokens."""
import math

import numpy as np
import pytest
import torch

import layers_ref as ref
import paged_hybrid_sliding_gb300 as phs
import synth
from gpu_util import dev

pytestmark = pytest.mark.gpu

CHUNK, TABLE, SHORT = 128, 536, 16


# ---------------------------------------------------------------- workspaces --
@pytest.mark.parametrize("B,H,P,N,total,most", [
    (65535, 128, 64, 64, 70_000, 100),          # 4.5e9 floats of tables
    (65535, 64, 64, 128, 65535 * 17, 17),       # 2.5e9: negative as a 32-bit number
    (2000, 4096, 64, 64, 34_000, 17),
    (16, 64, 64, 128, 32_000, 2000)])
def test_workspace_holds_a_table_for_each_chunk_and_head(B, H, P, N, total, most):
    """(The size alone: nothing is launched.)  Plans without segments hold the
    tables and nothing else, rounded up to 256 bytes."""
    want = (total // CHUNK + B + 1) * H * TABLE * 4
    got = phs.scan_prompt_workspace_bytes(B, H, 1, P, N, total, most)
    assert want <= got <= want + 256
