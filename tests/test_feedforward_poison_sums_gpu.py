"""Few rows, routing and the gradients on the debug copy of the library whose kernels fill their LDS
with NaN, and with what is past any index: their sums, keys and slots in LDS are all written before they
are read, so the copy's results are the library's to the bit."""
import ctypes
import os

import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from dense_fp16_gemm_f16_amd import build, segments
from tests import _feedforward as ref

pytestmark = pytest.mark.gpu
F16, F32, INF, NAN = torch.float16, torch.float32, float("inf"), float("nan")


@pytest.fixture
def same(monkeypatch):
    """Calls on the library and then on its copy; their results are equal."""
    if not os.path.exists(build.POISON_LIB):
        pytest.skip("libgemm_f16_poison.so is not built")
    copy = g._declare(ctypes.CDLL(build.POISON_LIB))

    def check(*calls):
        want = [c() for c in calls]
        torch.cuda.synchronize()
        with monkeypatch.context() as m:
            m.setattr(g, "_lib", copy)
            segments._workspace_bytes.cache_clear()
            got = [c() for c in calls]
            torch.cuda.synchronize()
        segments._workspace_bytes.cache_clear()
        for w, h in zip(want, got):
            for x, y in zip(w if isinstance(w, tuple) else (w,), h if isinstance(h, tuple) else (h,)):
                assert x is y is None or torch.equal(x, y)

    return check


@pytest.mark.parametrize("m,n,k", [(1, 100, 300), (2, 100, 4096), (3, 40, 8), (16, 250, 1001), (20, 1000, 512), (40, 4096, 1024), (64, 1024, 512)])
def test_few_rows(same, m, n, k):
    print("case: poisoned few rows", m, n, k, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    a, b, bias, res = ref.normal(gen, m, k), ref.normal(gen, n, k, std=k**-0.5), ref.normal(gen, n), ref.normal(gen, m, n)
    same(lambda: g.gemm_f16_fused_nt(a, b, bias, act="silu", residual=res, return_pre=True),
         lambda: g.gemm_f16_fused_nt(a, b, out_dtype=F32))


@pytest.mark.parametrize("experts,groups", [(8, 1), (8, 2), (20, 1), (40, 8), (64, 8), (128, 1), (160, 8), (256, 1), (256, 8), (256, 64), (300, 20),
                                            (512, 8), (1024, 1), (2048, 64)])
@pytest.mark.parametrize("what", ["normal", "alike", "masked"])
def test_routing(same, experts, groups, what):
    """alike: more candidates than a token has lanes, and keys and groups that are told apart in 64 bits."""
    print("case: poisoned routing", experts, groups, what, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(experts + groups)
    logits = torch.randn(67, experts, generator=gen, device="cuda")
    if what == "alike":
        logits = 0.75 + torch.randint(-2, 3, logits.shape, generator=gen, device="cuda") * 2.0**-23
    elif what == "masked":
        logits[torch.rand(logits.shape, generator=gen, device="cuda") < 0.7] = -INF
        logits[3], logits[4, ::2], logits[5, 1:] = NAN, NAN, -INF
    bias = torch.randn(experts, generator=gen, device="cuda") * (0.1 if what == "normal" else 2.0**-24)
    top = 1 if groups == 1 else max(1, groups // 2)
    most = experts // groups * top
    for fan in sorted({1, min(2, most), min(8, most), min(16, most), min(17, most), min(32, most)}):
        dg = torch.randn(67, fan, generator=gen, device="cuda")
        for score in ("softmax", "sigmoid"):
            ids, _ = g.route(logits, fan, score=score)
            same(*[lambda b=b, top2=top2: g.route(logits, fan, score=score, bias=b, groups=groups, top_groups=top, group_top=top2)
                   for b in (None, bias) for top2 in ((1, 2) if groups > 1 else (1,))],
                 lambda: g.route(logits, fan, score=score, renormalize=False),
                 lambda: g.route_grad(logits, ids, dg, score=score, renormalize=False))


@pytest.mark.parametrize("m,n", [(1, 7), (5, 4096), (33, 40), (64, 130), (300, 264), (777, 24), (5000, 1003)])
def test_gradient_of_the_activation(same, m, n):
    print("case: poisoned gradient", m, n, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    dy, pre = ref.normal(gen, m, n), ref.normal(gen, m, n, std=2.0)
    same(lambda: g.gemm_f16_fused_grad(dy, pre, act="gelu"), lambda: g.gemm_f16_fused_grad(dy.float()))


@pytest.mark.parametrize("tokens,fan,n", [(1, 1, 1), (1, 2, 4096), (5, 1, 1500), (40, 3, 100), (17, 11, 2056), (300, 4, 1032), (64, 2, 3001)])
def test_combination(same, tokens, fan, n):
    print("case: poisoned combination", tokens, fan, n, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(tokens + n)
    ids = torch.randint(-1, 6, (tokens, fan), generator=gen, device="cuda", dtype=torch.int32)
    _, inverse, offsets = g.group_rows(ids, 6)
    rows, dy = ref.normal(gen, tokens * fan, n), ref.normal(gen, tokens, n)
    gates = torch.rand(tokens, fan, generator=gen, device="cuda")
    same(lambda: g.combine_rows_grad(dy, rows, inverse, offsets, gates), lambda: g.combine_rows(rows, inverse, offsets, fan, gates=gates),
         lambda: g.group_rows(ids, 6))
