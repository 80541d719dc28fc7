"""What adapters keep of an inner product h = scale (x D^T): all of its fp32
bits and its infinities, at every row count."""
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _segments as ref

pytestmark = pytest.mark.gpu


def _call(x, w, down, up, ids, scale=None):
    order, _, off = g.group_rows(ids, down.shape[0])
    return g.gemm_f16_lora_nt(x, w, down, up, ids, order, off, scale)


def _one_adapter(rows, n, k, rank):
    z = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    return z(rows, k), z(n, k), z(1, rank, k), z(1, n, rank), torch.zeros(rows, dtype=torch.int32, device="cuda")


# few rows; aligned tiles, rank a multiple of 4 and not; rows that are not 16-byte aligned
FORMS = [(6, 40, 64, 16), (70, 40, 64, 16), (300, 264, 64, 32), (600, 520, 128, 64), (300, 130, 64, 18), (90, 61, 75, 16)]


@pytest.mark.parametrize("rows, n, k, rank", FORMS)
def test_an_infinite_inner_product_gives_what_fp32_gives(rows, n, k, rank):
    """h = +-inf in one rank: y = h u there, so +-inf, and NaN where u is 0."""
    gen = torch.Generator(device="cuda").manual_seed(rank)
    x, w, down, up, _ = _one_adapter(rows, n, k, rank)
    down, up = down.repeat(2, 1, 1), up.repeat(2, 1, 1)
    ids = torch.randint(-1, 2, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    for t in (x, w, down, up):
        t.copy_(ref.eighths(gen, *t.shape))
    x[:, 5] = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.5, 1.0, -1.0).half()
    down[1, 3, 5] = float("inf")
    up[1, :, 3] = (torch.arange(n, device="cuda") % 5 - 2).half() * 0.375  # both signs, of one and two bf16 parts, and 0
    up[1, n // 2:, 3] *= 1.0009765625
    out = _call(x, w, down, up, ids).cpu()
    want, err = ref.lora(*(t.cpu() for t in (x, w, down, up, ids)), None)
    wild = ~torch.isfinite(want)
    assert wild[ids.cpu() == 1].all() and not wild[ids.cpu() != 1].any()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[wild].nan_to_num(1.0), want[wild].half().nan_to_num(1.0))
    assert ref.worst(out[~wild], want[~wild], err[~wild], torch.float16) <= 1.0


@pytest.mark.parametrize("rows, n, k, rank", FORMS)
def test_the_largest_inner_product_times_zero_is_zero(rows, n, k, rank):
    x, w, down, up, ids = _one_adapter(rows, n, k, rank)
    x[:, 0], w[:, 0], down[0, :, 0] = 1.0, 2.0, 1.0
    down[0, 1, 0] = -1.0
    scale = torch.full((1,), torch.finfo(torch.float32).max, device="cuda")
    assert (_call(x, w, down, up, ids, scale) == 2.0).all()


@pytest.mark.parametrize("rows, n, k, rank", FORMS)
def test_every_bit_of_an_inner_product_counts(rows, n, k, rank):
    """Pairs of ranks with h and h + d, h of 19 bits, and u = -1 and 1: y is the
    sum of the d, and every partial sum is a whole number below 2^24."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, w, down, up, ids = _one_adapter(rows, n, k, rank)
    x[:, 0], x[:, 1] = 4096.0, 1.0
    x[:, 2] = torch.randint(-2, 3, (rows,), generator=gen, device="cuda").half()
    pairs = min(rank // 2, 8)
    high = torch.randint(0, 128, (pairs,), generator=gen, device="cuda").half()
    low = torch.randint(0, 2048, (pairs,), generator=gen, device="cuda").half()
    d = torch.randint(-3, 4, (pairs,), generator=gen, device="cuda").half()
    down[0, 0:2 * pairs:2, 0] = down[0, 1:2 * pairs:2, 0] = high
    down[0, 0:2 * pairs:2, 1] = down[0, 1:2 * pairs:2, 1] = low
    down[0, 1:2 * pairs:2, 2] = d
    up[0, :, 0:2 * pairs:2], up[0, :, 1:2 * pairs:2] = -1.0, 1.0
    want = x[:, 2] * d.sum()
    assert torch.equal(_call(x, w, down, up, ids), want[:, None].expand(rows, n))


def test_every_bit_of_a_single_inner_product():
    """2^23 + 2^12 + 1 against -2^23 and -2^12."""
    for rows, n, k, rank in FORMS:
        x, w, down, up, ids = _one_adapter(rows, n, k, rank)
        x[:, 0], x[:, 1] = 4096.0, 1.0
        x[:, 2] = 1.0
        down[0, 0, 0], down[0, 0, 1], down[0, 0, 2] = 2048.0, 1.0, 4096.0
        down[0, 1, 0], down[0, 2, 0] = 2048.0, 1.0
        up[0, :, 0], up[0, :, 1], up[0, :, 2] = 1.0, -1.0, -1.0
        assert (_call(x, w, down, up, ids) == 1.0).all(), (rows, n, k, rank)


@pytest.mark.parametrize("rows, n, k, rank", FORMS)
def test_adapters_are_as_exact_as_fp32(rows, n, k, rank):
    """The bound of sums in fp32: k terms and a scale for h, then k + 5 rank
    terms, and the least product of parts, below 2^-23 of its term."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    x, w, down, up, ids = _one_adapter(rows, n, k, rank)
    for t in (x, w, down, up):
        t.copy_(ref.normal(gen, *t.shape))
    up[0, :, 1::2] = -up[0, :, ::2][:, :rank // 2]  # pairs of ranks that nearly cancel
    down[0, 1::2] = down[0, ::2][:rank // 2]
    down[0, 1::2, 0] += 2.0**-9
    w.zero_()
    scale = torch.full((1,), 0.75, device="cuda")
    want, _ = ref.lora(x, w, down, up, ids, scale)
    h = 0.75 * torch.mm(x.double().abs(), down[0].double().abs().T.contiguous())
    mag = torch.mm(h, up[0].double().abs().T.contiguous())
    assert ref.worst(_call(x, w, down, up, ids, scale), want, mag * (2 * k + 6 * rank + 4) * 2.0**-23, torch.float16) <= 1.0


def _many_adapters(rows, adapters, rank, n, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(-1, adapters, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    make = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda").half()  # noqa: E731
    t = [make(rows, k), make(n, k), make(adapters, rank, k), make(adapters, n, rank)]
    return t, ids


@pytest.mark.parametrize("rows, adapters, rank, n, k", [(300, 37, 64, 264, 64), (1000, 200, 32, 512, 64), (500, 40, 100, 136, 72),
                                                        (260, 100, 48, 130, 33), (60, 64, 64, 200, 72)])
def test_adapters_many_to_a_tile_are_exact(rows, adapters, rank, n, k):
    """Sums that are exact in fp32 come out exact: zeros too."""
    t, ids = _many_adapters(rows, adapters, rank, n, k, rows)
    order, _, off = g.group_rows(ids, adapters)
    want, _ = ref.lora(*t, ids, None)
    assert float(want.abs().max()) <= 2048  # whole numbers that fp16 holds
    assert torch.equal(g.gemm_f16_lora_nt(*t, ids, order, off), want.half())


@pytest.mark.parametrize("rows, n, k, rank", FORMS)
def test_an_infinite_inner_product_meets_an_infinite_weight(rows, n, k, rank):
    """inf * inf is inf: not what 0 or a finite stand-in for either gives."""
    x, w, down, up, ids = _one_adapter(rows, n, k, rank)
    x[:, 0], w[:, 0] = 1.0, 2.0
    down[0, :, 0] = 0.5
    down[0, 2, 0] = float("inf")
    up[0] = 0.25
    up[0, :, 2] = float("inf")
    up[0, 1::2, 2] = float("-inf")
    x[rows // 2:, 0] = -1.0
    out = _call(x, w, down, up, ids)
    sign = x[:, :1].float() * torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0)
    assert torch.equal(out.float(), sign * float("inf"))
