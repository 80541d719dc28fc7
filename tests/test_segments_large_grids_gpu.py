"""Segmented products whose tiles need more than the 2^32 threads that one
launch can have along its grid."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _segments as ref

pytestmark = pytest.mark.gpu


def test_weight_gradient_of_more_tiles_than_a_launch_holds():
    """2^20 groups of 1 x 2176: 17 tiles each, 4.6 GB of results."""
    groups, n, k = 1 << 20, 2176, 1
    gen = torch.Generator(device="cuda").manual_seed(2)
    at = [0, 5, 5, 400_000, groups - 2, groups - 1]
    sizes = torch.zeros(groups, dtype=torch.int64)
    for s in at:
        sizes[s] += 1
    off = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).to(torch.int32).cuda()
    a, b = ref.eighths(gen, len(at), k), ref.eighths(gen, len(at), n)
    out = torch.full((groups, k, n), 3.0, dtype=torch.float16, device="cuda")
    g.gemm_f16_grouped_tn(a, b, off, out=out)
    for s in sorted(set(at)):
        rows = [r for r, q in enumerate(at) if q == s]
        assert torch.equal(out[s, 0], (a[rows].double() * b[rows].double()).sum(0).half())
        out[s] = 0
    for part in out.view(16, -1):
        assert not part.any()
