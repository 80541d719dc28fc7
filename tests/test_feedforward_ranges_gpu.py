"""The feed-forward layer's operators where a value leaves the range of its type."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _feedforward as ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
F16, F32 = torch.float16, torch.float32


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("m", [2, 40, 300])
def test_gradient_where_pre_is_an_infinity(act, m):
    """z past fp16's range, either sign: c is what the formula gives, pre an infinity, and the slope
    its limit.  A slope of 1 is off by at most the roundings of 1 - tail and of a reciprocal, below 2^-22, so
    dy (eighths) times it rounds to dy in fp16; up to 300 such terms of up to 1 have partial sums below 2^9,
    each of whose roundings is at most 2^-16: their sum is off by less than 300 (2^-22 + 2^-16) < 2^-7."""
    print("case: gradient past fp16's range", act, m, flush=True)
    n = 72
    # z = 65504 + x, past 65520, where fp16 ends
    x = torch.tensor([32.0, 4496.0, 65504.0], device="cuda")[torch.arange(m, device="cuda") % 3].to(F16)
    sign = torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0).to(F16)
    a = torch.zeros(m, 64, dtype=F16, device="cuda")
    b = torch.zeros(n, 64, dtype=F16, device="cuda")
    a[:, 0], a[:, 1] = 65504.0, x
    b[:, 0] = b[:, 1] = sign
    z = a.double() @ b.double().T
    got, pre = g.gemm_f16_fused_nt(a, b, act=act, return_pre=True, out_dtype=F32)
    assert torch.equal(pre, (sign.float() * INF).half().expand(m, n))
    assert torch.allclose(got.double(), ref.act(act, z), rtol=2.0**-20, atol=0.0)
    assert not bool(torch.isnan(g.gemm_f16_fused_nt(a, b, act=act)).any())
    gen = torch.Generator(device="cuda").manual_seed(m)
    slope = torch.ones(m, n, dtype=F16, device="cuda") if act is None else (sign > 0).to(F16).expand(m, n)
    for dy_type in (F16, F32):
        dy = ref.eighths(gen, m, n).to(dy_type)
        dz, dbias = g.gemm_f16_fused_grad(dy, pre if act else None, act=act)
        assert torch.equal(dz.half(), dy.half() * slope)
        assert torch.allclose(dbias.double(), (dy.double() * slope.double()).sum(0), rtol=0.0, atol=2.0**-7)


@pytest.mark.parametrize("act", ref.ACTS[1:])
def test_gradient_at_infinities_and_nan(act):
    """An infinite pre gives the slope's limit, a NaN a NaN, and neither touches the columns beside it."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    pre, dy = ref.normal(gen, 50, 43), torch.ones(50, 43, dtype=F16, device="cuda")
    want, _ = g.gemm_f16_fused_grad(dy, pre, act=act)
    pre[3, 5], pre[4, 42], pre[5, 41] = INF, -INF, NAN
    want[3, 5], want[4, 42] = 1.0, 0.0
    dz, dbias = g.gemm_f16_fused_grad(dy, pre, act=act)
    assert bool(torch.isnan(dz[5, 41])) and int(torch.isnan(dz).sum()) == 1
    assert int(torch.isnan(dbias).sum()) == 1 and bool(torch.isnan(dbias[41]))
    dz[5, 41] = want[5, 41]
    assert torch.equal(dz, want)
