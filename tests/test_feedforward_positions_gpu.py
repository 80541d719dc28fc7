"""Where in the batch a row stands makes no difference to its results: equal rows in every block of
64 give equal results to the bit, on random data, whose sums depend on their order."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _feedforward as ref

pytestmark = pytest.mark.gpu
F16, F32 = torch.float16, torch.float32


# the ring with few columns and few rows, undivided (K-tiles a multiple of 8, not, fewer than 8) and in parts;
# one and two rows, few rows, tiles with fewer and with more of them than CUs, rows that are not 16-byte aligned
@pytest.mark.parametrize("m,n,k", [(16384, 64, 4096), (16384, 64, 4160), (20000, 64, 1032), (8192, 64, 2056), (70000, 24, 448),
                                   (1024, 64, 4096), (5000, 24, 4096), (64, 16384, 4096), (50, 20000, 1000), (64, 4096, 4096),
                                   (48, 4096, 4096), (130, 264, 2056), (2, 1000, 4096), (20, 1000, 512), (1000, 1000, 1000),
                                   (4352, 4096, 256), (3000, 4104, 1032), (4096, 320, 999), (128, 512, 4099)])
def test_equal_rows_give_equal_results(m, n, k):
    print("case: equal rows", m, n, k, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, b = ref.normal(gen, min(m, 64), k), ref.normal(gen, n, k, std=k**-0.5)
    rows = torch.arange(m, device="cuda") % len(a)
    batch = a[rows].contiguous()
    for out_type in (F16, F32):
        c = g.gemm_f16_fused_nt(batch, b, out_dtype=out_type)
        assert torch.equal(c, c[:len(a)][rows])
    y, _, err, _ = ref.fused(batch, b, None, None, None)
    assert ref.worst(c, y, err, F32) <= 1
