"""The cache policies of the walking products' stores: past 256 MiB, rows of whole 128-byte lines and
rows that are not, on each of the walked tiles."""
import os

import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _codeobj
from tests import _feedforward as ref

F16 = torch.float16


def test_every_policy_is_built_for_every_walked_tile():
    if not os.path.exists(g.LIB_PATH):
        pytest.fail(f"{g.LIB_PATH} is not built")
    names = [r[".name"] for r in _codeobj.kernel_records(g.LIB_PATH) if "fused_walk_kernel" in r[".name"]]
    for bm, bn in ((256, 256), (256, 128), (128, 256)):
        for act, residual in [(a, 0) for a in range(5)] + [(0, 1)]:
            for policy in range(3):
                assert sum(f"CfgILi{bm}ELi{bn}E" in n and f"ELi{act}ELb{residual}ELi{policy}ELb" in n for n in names) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("tile,m,n,k", [("256x256", 33000, 4104, 512), ("256x256", 33000, 4096, 512), ("256x128", 60000, 2056, 200),
                                        ("256x128", 40000, 2056, 256), ("128x256", 30000, 4104, 192), ("128x256", 30000, 4096, 192)])
def test_walked_tiles_past_the_cache(tile, m, n, k):
    """Sums of eighths, exact in fp32 in any order."""
    print("case: store policies", tile, m, n, k, flush=True)
    assert g.select_tile(m, n, k) == getattr(g, "TILE_" + tile) and (m + n) * k * 2 + 4 * m * n > 256 << 20
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    a, b = ref.eighths(gen, m, k), ref.eighths(gen, n, k)
    bias, res = ref.eighths(gen, n), ref.eighths(gen, m, n)
    z = (a.float() @ b.float().T).add_(bias.float())
    buf = torch.full((m * n + 128,), 7.0, dtype=F16, device="cuda")
    for start in (64, 72):  # on a line, and not
        out = buf[start:start + m * n].view(m, n)
        got, pre = g.gemm_f16_fused_nt(a, b, bias, act="relu", return_pre=True, out=out)
        assert torch.equal(out, z.clamp(min=0).to(F16)) and torch.equal(pre, z.to(F16))
        g.gemm_f16_fused_nt(a, b, bias, residual=res, out=out)
        assert torch.equal(out, (z + res.float()).to(F16))
        assert bool((buf[:start] == 7).all()) and bool((buf[start + m * n:] == 7).all())
        buf.fill_(7.0)
