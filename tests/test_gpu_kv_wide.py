"""Attention over the caches on the GPU for heads above 128, few rows: one CTA an SM (16-bit caches), two (8 bits).
(That these are resident is asserted where kv_token.cuh compiles.)"""

import numpy as np
import pytest
import torch

from test_gpu_kv import _call, _check, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H", [144, 256])
@pytest.mark.parametrize("B, Nq, Nkv, S", [(24, 16, 8, 1), (90, 4, 2, 4), (3, 16, 8, 1), (200, 6, 3, 1)])
def test_wide_heads_of_ragged_sequences(lib, cuda, fp8, H, B, Nq, Nkv, S):
    """Clusters, work dealt to the CTAs that are resident, a CTA for each problem; without a workspace too."""
    rng = np.random.default_rng(B)
    L = 500
    past = np.where(rng.random(B) < 0.3, rng.integers(-S, 2, B), rng.integers(0, L - S + 1, B))
    past[0], past[-1] = L - S, 0
    a = _make(61, "bf16", B, S, Nq, Nkv, H, L, past.tolist(), fp8, cap=9.0)
    first = _check(lib, a, cuda)
    assert lib.last_kernel() == "kv_token_kernel" and torch.equal(_call(lib, a, cuda), first)
    _check(lib, a, cuda, workspace=torch.empty(0, dtype=torch.uint8, device=cuda))
