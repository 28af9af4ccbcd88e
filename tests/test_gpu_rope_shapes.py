"""Norm + rotation where its launch changes shape: around as many tokens as are resident at once,
with and without a cache, against 64 bits."""
import numpy as np
import pytest
import torch

import _q4
from test_gpu_serving_inputs import _rope_case, _rope_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,dim,tokens", [
    (24, 4, 256, (75, 76, 77, 87, 88)), (32, 8, 256, (50, 51, 52, 61)), (12, 2, 256, (152, 153)),
    (24, 4, 128, (151, 152, 153)), (16, 4, 64, (303, 304, 305)), (70, 3, 256, (32, 33, 600))])
def test_rope_where_the_launch_changes_shape(cuda_lib, hq, hkv, dim, tokens):
    pa = cuda_lib
    for T in tokens:
        q, k, v, w, table, pos = _rope_case(T, hq, hkv, dim, 64, seed=T)
        qo, ko = pa.qk_norm_rope(q, k, w[0], w[1], table, pos, 1e-6)
        for got, x, weight in ((qo, q, w[0]), (ko, k, w[1])):
            ref, tol = _rope_ref(x, weight, table, pos, False)
            assert (np.abs(_q4.f64(got) - ref) <= tol).all(), T
        # bit for bit what the call with the write gives
        kv = torch.zeros(T, 2, 1, hkv, dim, dtype=torch.bfloat16, device="cuda")
        slots = torch.arange(T, device="cuda").flip(0).contiguous()
        qc = pa.qk_norm_rope_cache(q, k, v, w[0], w[1], table, pos, 1e-6, kv[:, 0], kv[:, 1], slots)
        assert torch.equal(qc, qo) and torch.equal(kv[:, 0, 0].flip(0), ko) and torch.equal(kv[:, 1, 0].flip(0), v), T
    assert pa.device_errors() == 0
