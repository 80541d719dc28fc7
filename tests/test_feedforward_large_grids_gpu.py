"""The feed-forward layer's operators at sizes that need more than the 2^32 threads that one
launch can have along its grid."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g

pytestmark = pytest.mark.gpu
F16 = torch.float16


def _counted(rows, k):
    """fp16 [rows, k], each row its number modulo 251 and zeros."""
    x = torch.zeros(rows, k, dtype=F16, device="cuda")
    x[:, 0] = torch.arange(rows, dtype=torch.int32, device="cuda").remainder_(251).to(F16)
    return x


@pytest.mark.parametrize("few", [False, True])
def test_product_of_more_tiles_than_a_launch_holds(few):
    """2^30 - 1 rows of one column, and one row of 2^30 - 1 columns."""
    print("case: large grid, product", few, flush=True)
    many, k = (1 << 30) - 1, 8
    x, one = _counted(many, k), torch.zeros(1, k, dtype=F16, device="cuda")
    one[0, 0] = 2.0
    y = g.gemm_f16_fused_nt(one, x, act="relu") if few else g.gemm_f16_fused_nt(x, one, act="relu")
    assert torch.equal(y.view(-1), x[:, 0].mul_(2))


def test_routing_of_more_tokens_than_a_launch_holds():
    print("case: large grid, routing", flush=True)
    tokens = (1 << 28) + 3  # 16 a workgroup
    logits = torch.zeros(tokens, 2, dtype=F16, device="cuda")
    logits[1::2, 1] = 1.0
    ids, gates = g.route(logits, 1)
    assert torch.equal(ids.view(-1), torch.arange(tokens, dtype=torch.int32, device="cuda").remainder_(2))
    assert bool((gates == 1).all())
    assert not bool(g.route_grad(logits, ids, gates).any())  # the gate of one expert does not change


def test_combination_of_more_tokens_than_a_launch_holds():
    print("case: large grid, combination", flush=True)
    tokens = (1 << 29) + 40  # 32 a workgroup, of the gradient 4
    rows = _counted(tokens, 1)
    inverse = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    assert torch.equal(g.combine_rows(rows, inverse, offsets, 1), rows.flip(0))
    dy = torch.full((tokens, 1), 2.0, dtype=F16, device="cuda")
    gates = torch.full((tokens, 1), 0.5, device="cuda")
    drows, dgates = g.combine_rows_grad(dy, rows, inverse, offsets, gates)
    assert bool((drows == 1).all())
    assert torch.equal(dgates, rows.flip(0).float().mul_(2))
