"""Segmented products with far more groups than rows, and grids past the
2^32 threads of one launch: sizes inside the documented limits are served."""
import numpy as np
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _segments as ref

pytestmark = pytest.mark.gpu

MOST = 1 << 20  # groups


def _zeros(*shape):
    return torch.zeros(*shape, dtype=torch.float16, device="cuda")


def _offsets(at, groups, rows):
    """Row r in group at[r] (rising), rows behind the last of them in no group."""
    sizes = np.zeros(groups, dtype=np.int64)
    np.add.at(sizes, np.asarray(at, dtype=np.int64), 1)
    assert len(at) <= rows
    return ref.offsets_of(sizes).cuda()


@pytest.mark.parametrize("at, tail", [([0], 0), ([MOST - 1], 0), ([70001, 70001, 70001, 900000], 3), ([], 2)])
def test_few_rows_in_most_groups(at, tail):
    """17 GB of weights, few of them read."""
    n, k, gen = 1024, 8, torch.Generator(device="cuda").manual_seed(1)
    b = _zeros(MOST, n, k)
    for s in set(at):
        b[s] = ref.eighths(gen, n, k)
    rows = len(at) + tail
    a, off = ref.eighths(gen, rows, k), _offsets(at, MOST, rows)
    out = g.gemm_f16_grouped_nt(a, b, off)
    for r, s in enumerate(at):
        assert torch.equal(out[r], (b[s].double() @ a[r].double()).half())
    assert not out[len(at):].any()


@pytest.mark.parametrize("groups", [3, 63, 64, 65, 500, 4097])
@pytest.mark.parametrize("n, k", [(40, 72), (33, 35)])
def test_fewer_rows_than_groups(groups, n, k):
    gen = torch.Generator(device="cuda").manual_seed(groups)
    for rows in (1, 2, min(groups, 40)):
        at = torch.randint(0, groups, (rows,), generator=gen, device="cuda").sort().values.tolist()
        at = [at, at[: rows // 2], [groups - 1] * rows, [0] * rows][rows % 4]
        a, b, off = ref.eighths(gen, rows, k), ref.eighths(gen, groups, n, k), _offsets(at, groups, rows)
        want, _, _ = ref.grouped("nt", a, b, off.tolist())
        assert torch.equal(g.gemm_f16_grouped_nt(a, b, off), want.half())


@pytest.mark.parametrize("offsets", [[0] + [9, -5, 1 << 30] * 33, [5] * 100, list(range(99, -1, -1)), [-1] * 100])
@pytest.mark.parametrize("n, k", [(96, 80), (61, 75)])
def test_few_rows_with_offsets_that_break_the_rules(offsets, n, k):
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, b = ref.eighths(gen, 12, k), ref.eighths(gen, 99, n, k)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    whole = torch.full((12 * n + 4096,), 7.0, dtype=torch.float16, device="cuda")
    g.gemm_f16_grouped_nt(a, b, off, out=whole[2048:][:12 * n].view(12, n))
    assert (whole[:2048] == 7).all() and (whole[2048 + 12 * n:] == 7).all()


@pytest.mark.parametrize("rows, k, rank, n", [(1, 8, 256, 8), (3, 16, 256, 8), (100, 9, 1024, 1)])
def test_most_adapters(rows, k, rank, n):
    """4 to 19 GB of adapters, one of them used."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    down, up = _zeros(MOST, rank, k), _zeros(MOST, n, rank)
    s = 777_777
    down[s], up[s] = ref.eighths(gen, rank, k), ref.eighths(gen, n, rank)
    x, w = ref.eighths(gen, rows, k), ref.eighths(gen, n, k)
    ids = torch.full((rows,), s, dtype=torch.int32, device="cuda")
    ids[1::2] = -1
    order = ids.argsort(descending=True, stable=True).to(torch.int32)
    off = torch.zeros(MOST + 1, dtype=torch.int32, device="cuda")
    off[s + 1:] = (rows + 1) // 2
    out = g.gemm_f16_lora_nt(x, w, down, up, ids, order, off)
    mine = torch.where(ids == s, 0, -1)
    want, err = ref.lora(x, w, down[s:s + 1], up[s:s + 1], mine, None)
    assert ref.worst(out, want, err, torch.float16) <= 1.0
