"""Indices, offsets and orders that break the rules, and gathers past 2 GiB, on
each kernel that a segmented product can run on: what is valid comes out right,
and nothing is written outside the output."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _segments as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _guarded(shape, dtype=torch.float16):
    count = 1
    for v in shape:
        count *= v
    whole = torch.full((count + 4096,), 7.0, dtype=dtype, device="cuda")

    def check():
        assert (whole[:2048] == 7).all() and (whole[2048 + count:] == 7).all()
    return whole[2048:][:count].view(shape), check


@pytest.mark.parametrize("k", [4096, 4095])
@pytest.mark.parametrize("sizes", [[30, 25], [150, 0, 90]])
def test_gather_past_two_gib_with_many_rows(sizes, k):
    """Too many rows a segment for the few-row kernel: operands staged through registers."""
    tokens, rows, gen = 600_000, sum(sizes), _gen(k)  # 4.9 GB
    a = torch.zeros(tokens, k, dtype=torch.float16, device="cuda")
    index = torch.randint(0, tokens, (rows,), generator=gen, device="cuda").to(torch.int32)
    index[:6] = torch.tensor([0, 262143, 262144, 524287, 524288, 599999], dtype=torch.int32)
    a[index.long()] = ref.eighths(gen, rows, k)
    b, off = ref.eighths(gen, len(sizes), 136, k), ref.offsets_of(sizes).cuda()
    want, _, _ = ref.grouped("nt", a[index.long()], b, off.tolist())
    assert torch.equal(g.gemm_f16_grouped_nt(a, b, off, index=index), want.half())


# few rows, the ring, whole tiles, the any-alignment kernel, walked tiles
SHAPES = [([3, 0, 9], 96, 80), ([60, 50, 0, 130], 320, 1024), ([200, 190], 512, 256), ([150, 0, 333], 257, 99),
          ([3000, 0, 700, 5, 4000], 2048, 1024), ([2500, 1200, 800, 4100], 1544, 200)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sizes, n, k", SHAPES)
def test_indices_outside_the_rows_read_zeros_on_every_kernel(sizes, n, k, f32):
    dtype = torch.float32 if f32 else torch.float16
    rows, fan, gen = sum(sizes) + 4, 3, _gen(n + k)
    tokens = rows // 2
    a, b, off = ref.eighths(gen, tokens, k), ref.eighths(gen, len(sizes), n, k), ref.offsets_of(sizes).cuda()
    index = torch.randint(0, tokens * fan, (rows,), generator=gen, device="cuda")
    bad = torch.rand(rows, generator=gen, device="cuda") < 0.3
    wild = torch.tensor([-1, tokens * fan, -(1 << 31), (1 << 31) - 1, tokens * fan + 2, -3], device="cuda")
    index = torch.where(bad, wild[torch.randint(0, 6, (rows,), generator=gen, device="cuda")], index).to(torch.int32)
    want, _, _ = ref.grouped("nt", a, b, off.tolist(), torch.where(bad, 0, index), fan)
    want[bad] = 0
    out, check = _guarded((rows, n), dtype)
    g.gemm_f16_grouped_nt(a, b, off, index=index, fan=fan, out_dtype=dtype, out=out)
    assert torch.equal(out, want.to(dtype))
    check()


BROKEN = [[0, -5, 1 << 30, 3, 700, -1], [9000, 6000, 3000, 0, 8000, 2], [0, 8000, 0, 8000, 0, 8000]]


@pytest.mark.parametrize("offsets", BROKEN)
@pytest.mark.parametrize("rows, n, k", [(7700, 2048, 1024), (2000, 1544, 200), (300, 320, 1024), (400, 257, 99), (40, 96, 80), (40, 61, 75)])
@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
def test_offsets_that_break_the_rules_stay_in_range_on_every_kernel(kind, rows, n, k, offsets):
    gen, groups = _gen(rows), 5
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    a = ref.eighths(gen, rows, k)
    b = ref.eighths(gen, rows, n) if kind == "tn" else ref.eighths(gen, groups, *((n, k) if kind == "nt" else (k, n)))
    out, check = _guarded((groups, k, n) if kind == "tn" else (rows, n))
    call = {"nt": g.gemm_f16_grouped_nt, "nn": g.gemm_f16_grouped_nn, "tn": g.gemm_f16_grouped_tn}[kind]
    call(a, b, off, out=out)
    check()
    if kind == "nt":
        index = torch.randint(-(1 << 31), 1 << 31, (rows,), generator=gen, device="cuda").to(torch.int32)
        call(a, b, off, index=index, fan=2, out=out)
        check()


@pytest.mark.parametrize("rows, n, k, rank", [(1, 96, 80, 8), (20, 96, 80, 7), (64, 130, 1000, 16), (70, 96, 80, 7), (300, 264, 512, 64),
                                              (300, 61, 75, 9), (90, 100, 5, 8), (1500, 520, 512, 33)])
def test_adapter_orders_and_offsets_that_break_the_rules_stay_in_range(rows, n, k, rank):
    gen, adapters = _gen(rows), 4
    x, w = ref.eighths(gen, rows, k), ref.eighths(gen, n, k)
    down, up = ref.eighths(gen, adapters, rank, k), ref.eighths(gen, adapters, n, rank)
    any32 = lambda *s: torch.randint(-(1 << 31), 1 << 31, s, generator=gen, device="cuda").to(torch.int32)  # noqa: E731
    for off in ([5, 900, -3, 60, 7], [0, 1 << 30, 0, 1 << 30, 2], [3, 2, 1, 0, -1]):
        out, check = _guarded((rows, n))
        g.gemm_f16_lora_nt(x, w, down, up, any32(rows), any32(rows), torch.tensor(off, dtype=torch.int32, device="cuda"), out=out)
        check()
