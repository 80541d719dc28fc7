"""The feed-forward layer's products on the debug copy of the library whose kernels fill
their LDS with NaN before the first load: an operand read from LDS that nothing wrote, a
K tail that does not land as zeros or a wait too few gives a NaN.
"""
import ctypes
import os

import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from dense_fp16_gemm_f16_amd import build, segments
from tests import _feedforward as ref

pytestmark = pytest.mark.gpu
F16, F32 = torch.float16, torch.float32


@pytest.fixture
def poisoned(monkeypatch):
    if not os.path.exists(build.POISON_LIB):
        pytest.skip("libgemm_f16_poison.so is not built")
    monkeypatch.setattr(g, "_lib", g._declare(ctypes.CDLL(build.POISON_LIB)))
    segments._workspace_bytes.cache_clear()
    yield
    segments._workspace_bytes.cache_clear()


# few rows; parts of K on either tile and on the ring, with K in whole and broken K-tiles; each block
# tile with fewer and with more tiles than CUs; rows that are not 16-byte aligned, undivided and in parts
@pytest.mark.parametrize("m,n,k", [(1, 100, 700), (5, 264, 1000), (48, 520, 520), (65, 64, 4096), (128, 512, 4104), (512, 512, 2048),
                                   (8192, 64, 2056), (1000, 24, 512), (700, 300, 1000), (1025, 1032, 200), (2049, 2056, 136),
                                   (4352, 4096, 256), (4352, 4096, 200), (4608, 4100, 192), (128, 512, 4097), (700, 301, 999),
                                   (1500, 1500, 333), (4100, 1000, 130)])
def test_poisoned_lds_reaches_no_result(poisoned, m, n, k):
    print("case:", "poisoned", m, n, k, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, b, bias = ref.eighths(gen, m, k), ref.eighths(gen, n, k), ref.eighths(gen, n)
    for out_type in (F16, F32):
        residual = ref.eighths(gen, m, n).to(out_type)
        y, z, _, _ = ref.fused(a, b, bias, None, residual)
        got, pre = g.gemm_f16_fused_nt(a, b, bias, residual=residual, return_pre=True, out_dtype=out_type)
        assert torch.equal(got, y.to(out_type)) and torch.equal(pre, z.to(F16))
