"""Routing with biases at the ends of fp32's range, masks of its lowest value among them, against the
definition in 64 bits."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _feedforward as ref

pytestmark = pytest.mark.gpu
F32 = torch.float32
INF, LOWEST = float("inf"), torch.finfo(torch.float32).min


def _same(logits, fan, **how):
    ids, gates = g.route(logits, fan, **how)
    w_ids, w_gates = ref.route(logits, fan, **how)
    assert torch.equal(ids.cpu().long(), w_ids)
    # scores of logits below 8 in magnitude: an exp, up to 64 terms of a sum and a quotient
    assert ref.worst(gates.cpu(), w_gates, (8 + 64 + 12) * 2 * ref.U * w_gates.abs() + 2.0**-126, F32) <= 1


@pytest.mark.parametrize("experts,groups", [(16, 4), (64, 8), (40, 8), (512, 8), (8, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_masked_by_the_lowest_value(experts, groups, group_top, score):
    """Every other group at fp32's lowest value: its experts come last, in their order, and are not left out."""
    print("case: lowest biases", experts, groups, group_top, score, flush=True)
    per = experts // groups
    gen = torch.Generator(device="cuda").manual_seed(experts)
    logits = torch.randn(37, experts, generator=gen, device="cuda").clamp(-7, 7)
    bias = torch.zeros(groups, per, device="cuda")
    bias[::2] = LOWEST
    bias = bias.view(-1)
    fan = min(32, max(2, experts * 3 // 4))
    for top_groups in (groups, groups // 2 + 1):
        f = min(fan, per * top_groups)
        _same(logits, f, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top)
    _same(logits, min(fan, per), score=score, bias=torch.full((experts,), LOWEST, device="cuda"), groups=groups, top_groups=1,
          group_top=group_top)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("experts,groups", [(16, 4), (64, 8), (40, 8), (512, 8)])
def test_sums_of_two_past_the_range(sign, experts, groups):
    """Groups whose two largest biases add up past fp32's range, either sign: told apart all the same."""
    per = experts // groups
    gen = torch.Generator(device="cuda").manual_seed(groups)
    logits = torch.randn(20, experts, generator=gen, device="cuda").clamp(-7, 7)
    for large in (1.9e38, 3.0e38):
        step = torch.randperm(groups, generator=torch.Generator().manual_seed(experts)).float().cuda() * 1e36
        bias = (sign * (large + step))[:, None].expand(groups, per).reshape(-1).contiguous()
        for top_groups in (1, 2):
            _same(logits, 3, score="sigmoid", bias=bias, groups=groups, top_groups=top_groups, group_top=2)
        bias[per] = INF  # one expert of the second group
        _same(logits, 3, score="sigmoid", bias=bias, groups=groups, top_groups=2, group_top=2)
