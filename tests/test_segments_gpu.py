"""The segmented products on the GPU against their definitions in 64 bits
(_segments.py derives the bounds): row grouping, products grouped by
expert, their gradients, and low-rank adapters."""
import ctypes
import os

import numpy as np
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from dense_fp16_gemm_f16_amd import build
from tests import _segments as ref

pytestmark = pytest.mark.gpu

CALL = {"nt": lambda *a, **k: g.gemm_f16_grouped_nt(*a, **k), "nn": lambda *a, **k: g.gemm_f16_grouped_nn(*a, **k),
        "tn": lambda *a, **k: g.gemm_f16_grouped_tn(*a, **k)}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(kind, sizes, n, k, gen, make=ref.eighths, tail=0):
    rows = sum(sizes) + tail
    a = make(gen, rows, k)
    b = make(gen, rows, n) if kind == "tn" else make(gen, len(sizes), *((n, k) if kind == "nt" else (k, n)))
    return a, b, ref.offsets_of(sizes).cuda()


# ---- row grouping ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows, groups", [
    (0, 3), (1, 1), (1, 300), (63, 8), (64, 8), (65, 7), (128, 8), (1000, 1), (1025, 255), (4096, 256), (8191, 964),
    (8192, 64), (8193, 64), (20000, 13), (131072, 64), (131072, 2048), (300001, 1821)])
def test_group_rows(rows, groups, dtype):
    rng = np.random.default_rng(rows + groups)
    ids = rng.integers(-2, groups + 2, rows)  # some belong to no group
    ids[rng.random(rows) < 0.3] = 0           # and one group is large
    got = g.group_rows(torch.tensor(ids, dtype=dtype, device="cuda"), groups)
    for name, have, want in zip(("order", "inverse", "offsets"), got, ref.group_rows(ids, groups)):
        assert have.dtype == torch.int32
        assert np.array_equal(have.cpu().numpy(), want), name


@pytest.mark.parametrize("ids", [[5] * 200, [-1] * 200, list(range(200)), list(range(199, -1, -1))])
def test_group_rows_of_one_kind(ids):
    got = g.group_rows(torch.tensor(ids, device="cuda").view(20, 10), 200)
    for have, want in zip(got, ref.group_rows(ids, 200)):
        assert np.array_equal(have.cpu().numpy(), want)


def test_group_rows_takes_ids_past_32_bits():
    ids = torch.tensor([1 << 33, 1, -(1 << 33), 0, (1 << 32) + 1], device="cuda")
    order, _, offsets = g.group_rows(ids, 2)
    assert order.tolist() == [3, 1, 0, 2, 4] and offsets.tolist() == [0, 1, 2]


# ---- grouped products -----------------------------------------------------------

SIZES = [
    ([1], 8, 8), ([1], 1, 1), ([0, 1, 0], 5, 3), ([16] * 8, 128, 64), ([3, 0, 129, 64, 1], 136, 72),
    ([128, 256, 1], 256, 192), ([7, 5, 300, 0, 41], 131, 77), ([33, 100], 250, 1001), ([0, 0, 0], 64, 64),
    ([513, 0, 255], 520, 328), ([2] * 70, 72, 40), ([1, 0] * 64 + [200], 64, 136), ([20, 3], 1, 130), ([64], 129, 1),
    ([700, 90, 300], 384, 512), ([40, 24], 1000, 1024), ([9, 2], 96, 4096),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes, n, k", SIZES)
def test_grouped_is_exact_on_eighths(kind, sizes, n, k, f32):
    dtype = torch.float32 if f32 else torch.float16
    a, b, off = _inputs(kind, sizes, n, k, _gen(n * k))
    want, _, _ = ref.grouped(kind, a, b, off.tolist())
    out = CALL[kind](a, b, off, out_dtype=dtype)
    assert out.dtype == dtype and out.shape == want.shape
    assert torch.equal(out, want.to(dtype))


# more tiles than CUs (walked tiles, with a last round cut small, rows of no
# segment, one K-tile), long K on few tiles, and one row against wide weights
LARGE = [
    ([3000, 0, 700, 5, 4000], 2048, 1024, 300), ([2500, 1200, 800, 4100], 1544, 1608, 0), ([700, 300] * 8, 4096, 64, 0),
    ([60, 500, 0, 130], 4096, 4096, 0), ([1, 0, 2], 904, 3280, 1), ([9000], 2304, 200, 0), ([40, 0, 25, 30], 320, 4096, 9),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes, n, k, tail", LARGE)
def test_grouped_is_exact_at_large_sizes(kind, sizes, n, k, tail, f32):
    dtype = torch.float32 if f32 else torch.float16
    gen = _gen(n + k)
    a, b, off = _inputs(kind, sizes, n, k, gen, tail=tail)
    want, _, _ = ref.grouped(kind, a, b, off.tolist())
    assert torch.equal(CALL[kind](a, b, off, out_dtype=dtype), want.to(dtype))
    if kind == "nt":
        index = torch.randperm(3 * len(a), generator=gen, device="cuda")[:len(a)].to(torch.int32)
        want, _, _ = ref.grouped(kind, a, b, off.tolist(), index, 3)
        assert torch.equal(g.gemm_f16_grouped_nt(a, b, off, index=index, fan=3, out_dtype=dtype), want.to(dtype))


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes, n, k", [SIZES[i] for i in (3, 4, 5, 6, 14, 15)] + [s[:3] for s in LARGE[:5]])
def test_no_kernel_reads_lds_that_nothing_wrote(kind, sizes, n, k, monkeypatch):
    """The debug build fills LDS with NaN before the first load."""
    if not os.path.exists(build.POISON_LIB):
        pytest.skip("libgemm_f16_poison.so is not built")
    monkeypatch.setattr(g, "_lib", g._declare(ctypes.CDLL(build.POISON_LIB)))
    gen = _gen(n)
    a, b, off = _inputs(kind, sizes, n, k, gen)
    want, _, _ = ref.grouped(kind, a, b, off.tolist())
    assert torch.equal(CALL[kind](a, b, off), want.half())
    if kind == "nt":
        for rows, runs in ((3, False), (40, False), (300, True)):
            make = lambda gen, *s: torch.randint(-1, 2, s, generator=gen, device="cuda").half()  # noqa: E731
            x, w, down, up, ids, order, aoff, scale = _adapters(rows, 4, 16, n, min(k, 512), runs, gen, make)
            want, _ = ref.lora(x, w, down, up, ids, scale)
            assert torch.equal(g.gemm_f16_lora_nt(x, w, down, up, ids, order, aoff, scale), want.half())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sizes, n, k", [([900, 0, 31, 1500], 264, 520), ([5, 1, 2], 512, 2048), ([333, 250], 301, 1003),
                                         ([2500, 700, 1200, 600], 512, 1024)])
def test_grouped_on_random_operands(kind, sizes, n, k, f32):
    dtype = torch.float32 if f32 else torch.float16
    a, b, off = _inputs(kind, sizes, n, k, _gen(k), ref.normal)
    want, mag, terms = ref.grouped(kind, a, b, off.tolist())
    out = CALL[kind](a, b, off, out_dtype=dtype)
    assert ref.worst(out, want, mag * terms * 2.0**-23, dtype) <= 1.0


# ---- weight gradients of few tiles: each segment's rows in parts ------------------

SPLIT = [([9000], 256, 200, 0), ([16000], 64, 64, 5), ([0, 6000, 1, 63, 3000], 136, 264, 70), ([5000, 0, 4000], 61, 75, 0),
         ([2600, 2500], 513, 130, 3), ([64, 8000, 65], 8, 8, 0), ([3000, 900, 2000, 4000], 1024, 768, 0)]


@pytest.mark.parametrize("poisoned", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sizes, n, k, tail", SPLIT)
def test_split_weight_gradient_is_exact(sizes, n, k, tail, f32, poisoned, monkeypatch):
    if poisoned and not os.path.exists(build.POISON_LIB):
        pytest.skip("libgemm_f16_poison.so is not built")
    if poisoned:
        monkeypatch.setattr(g, "_lib", g._declare(ctypes.CDLL(build.POISON_LIB)))
    dtype = torch.float32 if f32 else torch.float16
    a, b, off = _inputs("tn", sizes, n, k, _gen(n + k), tail=tail)
    assert g.lib().gemm_f16_grouped_tn_workspace(len(a), len(sizes), n, k) >= 2 * 4 * len(sizes) * n * k
    want, _, _ = ref.grouped("tn", a, b, off.tolist())
    for offset in (0, 1, 8):  # the result at any alignment, nothing written beside it
        whole = torch.full((want.numel() + 600,), 7.0, dtype=dtype, device="cuda")
        out = whole[offset + 256:][:want.numel()].view(want.shape)
        g.gemm_f16_grouped_tn(a, b, off, out_dtype=dtype, out=out)
        assert torch.equal(out, want.to(dtype))
        assert (whole[:offset + 256] == 7).all() and (whole[offset + 256 + want.numel():] == 7).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n, k", [(264, 136), (75, 61)])
def test_split_weight_gradient_on_random_operands(n, k, f32):
    dtype = torch.float32 if f32 else torch.float16
    a, b, off = _inputs("tn", [4000, 31, 7000], n, k, _gen(k), ref.normal)
    want, mag, terms = ref.grouped("tn", a, b, off.tolist())
    out = g.gemm_f16_grouped_tn(a, b, off, out_dtype=dtype)
    assert ref.worst(out, want, mag * terms * 2.0**-23, dtype) <= 1.0
    assert torch.equal(out, g.gemm_f16_grouped_tn(a, b, off, out_dtype=dtype))  # the same bits again


def test_split_weight_gradient_keeps_segments_apart():
    sizes = [3000, 5000, 2000]
    a, b, off = _inputs("tn", sizes, 128, 72, _gen(3), tail=500)
    want, _, _ = ref.grouped("tn", a, b, off.tolist())
    a[3000:8000] = float("nan")
    b[10000:] = float("inf")
    out = g.gemm_f16_grouped_tn(a, b, off)
    assert torch.equal(out[[0, 2]], want[[0, 2]].half()) and torch.isnan(out[1]).all()


@pytest.mark.parametrize("offsets", [[0, 5000, 20, 9000], [0, -5, 1 << 30, 3], [7, 7, 7, 7], [9000, 6000, 3000, 0]])
def test_split_weight_gradient_with_offsets_that_break_the_rules(offsets):
    a, b, _ = _inputs("tn", [3000] * 3, 96, 80, _gen(1))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    whole = torch.full((3 * 80 * 96 + 4096,), 7.0, dtype=torch.float16, device="cuda")
    g.gemm_f16_grouped_tn(a, b, off, out=whole[2048:][:3 * 80 * 96].view(3, 80, 96))
    assert (whole[:2048] == 7).all() and (whole[2048 + 3 * 80 * 96:] == 7).all()


def test_split_weight_gradient_in_a_graph():
    a, b, off = _inputs("tn", [3000, 6000], 128, 256, _gen(9))
    g.gemm_f16_grouped_tn(a, b, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = g.gemm_f16_grouped_tn(a, b, off)
    for sizes in ([3000, 6000], [0, 9000], [8999, 1], [4000, 2000]):
        off.copy_(ref.offsets_of(sizes))
        a.copy_(ref.eighths(_gen(sizes[0]), *a.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, g.gemm_f16_grouped_tn(a, b, off))
        want, _, _ = ref.grouped("tn", a, b, off.tolist())
        assert torch.equal(out, want.half())


@pytest.mark.parametrize("fan", [1, 2, 3, 8])
@pytest.mark.parametrize("tokens, groups, n, k", [(1, 8, 64, 64), (50, 8, 136, 200), (333, 5, 257, 99), (700, 3, 256, 256),
                                                  (8, 8, 512, 2048)])
def test_grouped_nt_gathers_tokens(tokens, groups, n, k, fan):
    gen = _gen(tokens + fan)
    ids = torch.randint(-1, groups, (tokens, fan), generator=gen, device="cuda")
    order, _, off = g.group_rows(ids, groups)
    a, b = ref.eighths(gen, tokens, k), ref.eighths(gen, groups, n, k)
    want, _, _ = ref.grouped("nt", a, b, off.tolist(), order, fan)
    assert torch.equal(g.gemm_f16_grouped_nt(a, b, off, index=order, fan=fan), want.to(torch.float16))


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("n, k", [(128, 128), (61, 75), (256, 512)])
def test_rows_of_other_segments_do_not_reach_a_segment(kind, n, k):
    """NaN and infinities in the rows behind the last segment and in another
    segment stay there."""
    sizes = [70, 1, 300, 130]
    a, b, off = _inputs(kind, sizes, n, k, _gen(n), tail=200)
    ends = off.tolist()
    want, _, _ = ref.grouped(kind, a, b, ends)
    a[ends[2]:ends[3]] = float("nan")
    a[ends[4]:] = float("inf")
    if kind == "tn":
        b[ends[2]:ends[3]] = float("inf")
        b[ends[4]:] = float("nan")
    out = CALL[kind](a, b, off)
    if kind == "tn":
        keep = [0, 1, 3]
        assert torch.equal(out[keep], want[keep].half())
        assert torch.isnan(out[2]).all()
    else:
        for lo, hi in ((0, ends[2]), (ends[3], ends[4])):
            assert torch.equal(out[lo:hi], want[lo:hi].half())
        assert torch.isnan(out[ends[2]:ends[3]]).all()
        assert not out[ends[4]:].any()


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("n, k", [(64, 100), (33, 35), (256, 256)])
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_grouped_operands_at_any_offset_and_nothing_written_outside(kind, n, k, offset):
    """Operands and output inside larger buffers, `offset` elements from their
    start, with NaN around the operands and a pattern around the output."""
    sizes = [37, 0, 128, 5]
    a0, b0, off = _inputs(kind, sizes, n, k, _gen(offset))
    want, _, _ = ref.grouped(kind, a0, b0, off.tolist())
    a, b = (_inside(t, offset, float("nan")) for t in (a0, b0))
    for dtype in (torch.float16, torch.float32):
        whole = torch.full((want.numel() + 600,), 7.0, dtype=dtype, device="cuda")
        out = whole[offset + 200:][:want.numel()].view(want.shape)
        CALL[kind](a, b, off, out_dtype=dtype, out=out)
        assert torch.equal(out, want.to(dtype))
        assert (whole[:offset + 200] == 7).all() and (whole[offset + 200 + want.numel():] == 7).all()


def _inside(t, offset, fill):
    whole = torch.full((t.numel() + 512,), fill, dtype=t.dtype, device="cuda")
    v = whole[offset + 256:][:t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("kind", ["nt", "nn", "tn"])
@pytest.mark.parametrize("offsets", [[0, 500, 20, 90], [0, -5, 1 << 30, 3], [7, 7, 7, 7], [90, 60, 30, 0]])
def test_offsets_that_break_the_rules_stay_in_range(kind, offsets):
    """Unspecified values, but nothing outside the output (clamped offsets)."""
    a, b, _ = _inputs(kind, [30, 30, 30], 96, 80, _gen(1))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    shape = (3, 80, 96) if kind == "tn" else (90, 96)
    count = int(np.prod(shape))
    whole = torch.full((count + 4096,), 7.0, dtype=torch.float16, device="cuda")
    CALL[kind](a, b, off, out=whole[2048:][:count].view(shape))
    assert (whole[:2048] == 7).all() and (whole[2048 + count:] == 7).all()


@pytest.mark.parametrize("n, k", [(96, 80), (64, 2048)])
def test_an_index_outside_the_rows_reads_zeros(n, k):
    gen = _gen(5)
    a, b = ref.eighths(gen, 10, k), ref.eighths(gen, 2, n, k)
    index = torch.tensor([0, -1, 20, 19, 1 << 30, -(1 << 31), 3], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda")
    out = g.gemm_f16_grouped_nt(a, b, off, index=index, fan=2)
    ok = [0, 3, 6]
    want, _, _ = ref.grouped("nt", a[(index[ok] // 2).long()], b, [0, 2, 3])
    assert torch.equal(out[ok], want.half())
    assert not out[[1, 2, 4, 5]].any()


def test_an_index_into_no_rows_at_all():
    h = torch.empty(0, 1024, dtype=torch.float16, device="cuda")
    b = ref.eighths(_gen(1), 2, 64, 1024)
    index = torch.zeros(5, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    assert not g.gemm_f16_grouped_nt(h, b, off, index=index).any()
    assert not g.gemm_f16_grouped_nt(h[:, :7].contiguous(), b[:, :, :7].contiguous(), off, index=index).any()


def test_empty_extents():
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    h = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    assert g.gemm_f16_grouped_nt(h(0, 8), h(2, 8, 8), off).shape == (0, 8)
    assert g.gemm_f16_grouped_nn(h(0, 8), h(2, 8, 8), off).shape == (0, 8)
    out = torch.full((2, 8, 16), 3.0, dtype=torch.float16, device="cuda")
    assert not g.gemm_f16_grouped_tn(h(0, 8), h(0, 16), off, out=out).any()
    out = torch.full((5, 8), 3.0, dtype=torch.float16, device="cuda")
    assert not g.gemm_f16_grouped_nt(h(5, 0), h(2, 8, 0), off + 5, out=out).any()  # no terms: zeros
    assert g.gemm_f16_grouped_nt(h(5, 8), h(2, 0, 8), off).shape == (5, 0)


def test_gradients_against_differences():
    """<G, nt(X + D, W) - nt(X - D, W)> / 2 = <nn(G, W), D>, and the same by
    the weights: the product is linear, so the difference has no error of its
    own beyond the sums' rounding."""
    gen = _gen(8)
    sizes, n, k = [60, 0, 133, 9], 200, 168
    x, w, off = _inputs("nt", sizes, n, k, gen)
    up, dx, dw = ref.eighths(gen, sum(sizes), n), ref.eighths(gen, sum(sizes), k), ref.eighths(gen, len(sizes), n, k)
    f = lambda a, b: (g.gemm_f16_grouped_nt(a, b, off, out_dtype=torch.float32).double() * up.double()).sum()  # noqa: E731
    by_rows = g.gemm_f16_grouped_nn(up, w, off, out_dtype=torch.float32)
    by_weights = g.gemm_f16_grouped_tn(up, x, off, out_dtype=torch.float32)
    # eighths: every sum is exact, in fp16 as x +- dx too
    assert (f(x + dx, w) - f(x - dx, w)) / 2 == (by_rows.double() * dx.double()).sum()
    assert (f(x, w + dw) - f(x, w - dw)) / 2 == (by_weights.double() * dw.double()).sum()


def test_gather_past_two_gib():
    """Tokens beyond 2^31 bytes (and 2^32) into A."""
    k, tokens = 4096, 600_000  # 4.9 GB
    gen = _gen(2)
    a = torch.zeros(tokens, k, dtype=torch.float16, device="cuda")
    index = torch.tensor([0, 262143, 262144, 524287, 524288, 599999, 131072], dtype=torch.int32, device="cuda")
    a[index.long()] = ref.eighths(gen, len(index), k)
    b = ref.eighths(gen, 2, 72, k)
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")
    want, _, _ = ref.grouped("nt", a[index.long()], b, [0, 3, 7])
    assert torch.equal(g.gemm_f16_grouped_nt(a, b, off, index=index), want.half())


# ---- adapters -------------------------------------------------------------------

def _adapters(rows, adapters, rank, n, k, runs, gen, make=ref.eighths):
    ids = torch.randint(-1, adapters, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    if runs:
        ids = ids.sort(descending=True).values
    scale = 2.0 ** torch.randint(-2, 2, (adapters,), generator=gen, device="cuda").float()
    t = [make(gen, rows, k), make(gen, n, k), make(gen, adapters, rank, k), make(gen, adapters, n, rank)]
    order, _, off = g.group_rows(ids, adapters)
    return (*t, ids, order, off, scale)


ADAPTERS = [
    (1, 4, 16, 256, 256, False), (1, 1, 1, 8, 8, False), (3, 2, 4, 100, 77, False), (48, 32, 16, 512, 512, False),
    (16, 3, 12, 130, 136, False), (17, 5, 24, 264, 1000, True), (64, 64, 8, 128, 4096, False), (130, 6, 33, 300, 129, True),
    (200, 8, 64, 384, 256, False), (600, 5, 64, 520, 328, True), (300, 2, 100, 200, 64, True), (1000, 16, 16, 256, 128, False),
    (90, 3, 7, 61, 515, False), (2500, 4, 32, 256, 264, True), (4096, 8, 64, 1024, 1024, True), (700, 64, 16, 512, 512, False),
    (65, 2, 160, 300, 4096, False), (33, 3, 9, 100, 7, False), (130, 3, 9, 100, 5, False), (64, 4, 16, 2048, 9000, False),
    (300, 130, 8, 128, 256, False),
]


@pytest.mark.parametrize("rows, adapters, rank, n, k, runs", ADAPTERS)
@pytest.mark.parametrize("scaled", [True, False])
def test_lora(rows, adapters, rank, n, k, runs, scaled):
    x, w, down, up, ids, order, off, scale = _adapters(rows, adapters, rank, n, k, runs, _gen(rows + rank), ref.normal)
    scale = scale if scaled else None
    want, err = ref.lora(x, w, down, up, ids, scale)
    out = g.gemm_f16_lora_nt(x, w, down, up, ids, order, off, scale)
    # results past fp16's range round to infinity on both sides
    fits = want.abs() < 65000
    assert ref.worst(out[fits], want[fits], err[fits], torch.float16) <= 1.0


def test_lora_is_exact_on_small_whole_numbers():
    gen = _gen(4)
    make = lambda gen, *s: torch.randint(-1, 2, s, generator=gen, device="cuda").half()  # noqa: E731
    for rows, runs in ((5, False), (40, False), (333, False), (700, True)):
        x, w, down, up, ids, order, off, scale = _adapters(rows, 6, 16, 200, 256, runs, gen, make)
        want, _ = ref.lora(x, w, down, up, ids, scale)
        assert torch.equal(g.gemm_f16_lora_nt(x, w, down, up, ids, order, off, scale), want.half())


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_lora_keeps_an_inner_product_past_the_range_of_fp16(rows):
    """h = 2^20, y = 16 * 2^20 * 2^-14 + the shared part."""
    k, n, rank = 1024, 128, 16
    x = torch.full((rows, k), 32.0, dtype=torch.float16, device="cuda")
    w = torch.full((n, k), 2.0**-10, dtype=torch.float16, device="cuda")
    down = torch.full((2, rank, k), 32.0, dtype=torch.float16, device="cuda")
    up = torch.full((2, n, rank), 2.0**-14, dtype=torch.float16, device="cuda")
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ids[rows // 2:] = 1
    order, _, off = g.group_rows(ids, 2)
    out = g.gemm_f16_lora_nt(x, w, down, up, ids, order, off)
    assert (out == 32.0 + 16 * 64.0).all()


@pytest.mark.parametrize("rows", [6, 40, 300])
@pytest.mark.parametrize("where", ["down", "up", "x"])
def test_what_is_not_finite_stays_with_its_adapter(rows, where):
    x, w, down, up, ids, order, off, scale = _adapters(rows, 3, 16, 136, 264, False, _gen(rows), ref.eighths)
    ids[:3] = torch.tensor([0, 1, 2], dtype=torch.int32)
    order, _, off = g.group_rows(ids, 3)
    want, err = ref.lora(x, w, down, up, ids, scale)
    if where == "x":
        x[1, 5] = float("inf")
        hit = torch.arange(rows, device="cuda") == 1
    else:
        (down if where == "down" else up)[1, 2, 3] = float("nan")
        (down if where == "down" else up)[1, 1, 3] = float("inf")
        hit = ids == 1
    out = g.gemm_f16_lora_nt(x, w, down, up, ids, order, off, scale)
    assert ref.worst(out[~hit], want[~hit], err[~hit], torch.float16) <= 1.0
    assert not torch.isfinite(out[hit]).all(1).any()


def test_lora_orders_that_break_the_rules_stay_in_range():
    rows, n, k = 70, 96, 80
    x, w, down, up, ids, order, off, scale = _adapters(rows, 4, 8, n, k, False, _gen(1))
    order = torch.randint(-(1 << 31), 1 << 31, (rows,), generator=_gen(2), device="cuda").to(torch.int32)
    off = torch.tensor([5, 900, -3, 60, 7], dtype=torch.int32, device="cuda")
    whole = torch.full((rows * n + 4096,), 7.0, dtype=torch.float16, device="cuda")
    g.gemm_f16_lora_nt(x, w, down, up, ids, order, off, scale, out=whole[2048:][:rows * n].view(rows, n))
    assert (whole[:2048] == 7).all() and (whole[2048 + rows * n:] == 7).all()


# ---- streams, graphs, errors ----------------------------------------------------

def _step(x, w, ids, down, up, aids, fan=2):
    """Every operator once: a routed layer's forward and backward, and adapters."""
    order, inverse, off = g.group_rows(ids, w.shape[0])
    y = g.gemm_f16_grouped_nt(x, w, off, index=order, fan=fan)
    dx = g.gemm_f16_grouped_nn(y, w, off, out_dtype=torch.float32)
    dw = g.gemm_f16_grouped_tn(y, x[(order // fan).long()], off, out_dtype=torch.float32)
    aorder, _, aoff = g.group_rows(aids, down.shape[0])
    z = g.gemm_f16_lora_nt(x, w[0], down, up, aids, aorder, aoff)
    return order, inverse, off, y, dx, dw, z


def _state(tokens, seed):
    gen = _gen(seed)
    ids = torch.randint(0, 4, (tokens, 2), generator=gen, device="cuda", dtype=torch.int32)
    aids = torch.randint(-1, 3, (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    return [ref.normal(gen, tokens, 192), ref.normal(gen, 4, 256, 192, std=0.07), ids,
            ref.normal(gen, 3, 16, 192), ref.normal(gen, 3, 256, 16), aids]


@pytest.mark.parametrize("tokens", [5, 90, 700])
def test_graph_replays_match_eager(tokens):
    state = _state(tokens, 1)
    want = [[t.clone() for t in _step(*_state(tokens, s))] for s in range(1, 5)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(*state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(*state)
    for s in range(1, 5):
        for t, new in zip(state, _state(tokens, s)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        for have, expect in zip(out, want[s - 1]):
            assert torch.equal(have, expect)
        _step(*_state(tokens, 9))  # the program's own work between replays


def test_calls_on_another_stream():
    state = _state(300, 2)
    want = _step(*state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, w, ids = state[:3]
    order, inverse, off = g.group_rows(ids, 4, stream=side)
    y = g.gemm_f16_grouped_nt(x, w, off, index=order, fan=2, stream=side)
    dx = g.gemm_f16_grouped_nn(y, w, off, out_dtype=torch.float32, stream=side)
    side.synchronize()
    for have, expect in zip((order, inverse, off, y, dx), want):
        assert torch.equal(have, expect)


def test_the_same_call_gives_the_same_bits():
    for tokens in (5, 90, 700):
        state = _state(tokens, 3)
        first = [t.clone() for t in _step(*state)]
        for _ in range(3):
            for have, expect in zip(_step(*state), first):
                assert torch.equal(have, expect)


def test_refusals_on_the_gpu():
    h = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")    # noqa: E731
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_nt(h(4, 8), h(2, 8, 16), i(3))          # K differs
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_nt(h(4, 8), h(2, 8, 8), i(4))           # offsets of another count
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_nt(h(8, 4).T, h(2, 8, 8), i(3))         # not contiguous
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_nn(h(4, 8), h(2, 9, 8), i(3))
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_tn(h(4, 8), h(5, 8), i(3))              # row counts differ
    with pytest.raises(ValueError):
        g.gemm_f16_grouped_nt(h(4, 8), h(2, 8, 8), i(3), out=h(4, 9))
    with pytest.raises(TypeError):
        g.gemm_f16_grouped_nt(h(4, 8), h(2, 8, 8), torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(g.GemmError):
        g.gemm_f16_grouped_nt(h(4, 8), h(2, 8, 8), i(3), index=i(4), fan=0)
    with pytest.raises(g.GemmError):
        g.group_rows(i(4), 0)
    with pytest.raises(g.GemmError):
        a = h(4, 8)
        g.gemm_f16_grouped_nt(a, h(2, 8, 8), i(3), out=a)          # output over an input
    with pytest.raises(ValueError):
        g.gemm_f16_lora_nt(h(4, 8), h(8, 8), h(2, 4, 8), h(2, 8, 5), i(4), i(4), i(3))
