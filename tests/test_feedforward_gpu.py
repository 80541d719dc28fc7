"""The feed-forward layer's operators on the GPU against their definitions in 64
bits (tests/_feedforward.py), at the sizes, types and masks where they can go
wrong, and together as they are used."""
import ctypes

import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _feedforward as ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
F16, F32 = torch.float16, torch.float32


def _gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def _say(*what):
    print("case:", *what, flush=True)


def _offset(t, elements):
    """The same values, contiguous, starting `elements` into an allocation."""
    buf = torch.empty(t.numel() + elements + 8, dtype=t.dtype, device=t.device)
    view = buf[elements:elements + t.numel()].view(t.shape)
    view.copy_(t)
    return view


# ---- the product with its epilogue -----------------------------------------------

# one row, few rows, one tile, several tiles, more tiles than CUs; K below a chunk, odd, not a K-tile
SHAPES = [(1, 4096, 4096), (1, 1, 1), (1, 17, 7), (3, 40, 8), (16, 250, 1001), (17, 64, 264), (48, 1000, 520), (64, 72, 6000),
          (64, 9, 5), (65, 64, 4096), (100, 33, 3), (130, 520, 1000), (300, 520, 640), (257, 264, 72), (1000, 24, 512), (1025, 1032, 200),
          (700, 300, 999), (2049, 2056, 136), (4352, 4096, 256), (4608, 4100, 192), (5000, 3000, 64)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act", [None, "relu"])
def test_fused_exact_sums(m, n, k, act):
    """Multiples of 1/8: every sum is exact, so every path gives the one right answer, and pre too."""
    _say("fused exact", m, n, k, act)
    gen = _gen(m + n + k)
    a, b = ref.eighths(gen, m, k), ref.eighths(gen, n, k)
    for bias_type, out_type in ((None, F16), (F16, F32), (F32, F16)):
        bias = None if bias_type is None else ref.eighths(gen, n).to(bias_type)
        residual = None if bias_type is None else ref.eighths(gen, m, n).to(out_type)
        y, z, _, _ = ref.fused(a, b, bias, act, residual)
        got, pre = g.gemm_f16_fused_nt(a, b, bias, act=act, residual=residual, return_pre=True, out_dtype=out_type)
        assert torch.equal(got, y.to(out_type)), (bias_type, out_type)
        assert torch.equal(pre, z.to(F16))
        got = g.gemm_f16_fused_nt(a, b, bias, act=act, residual=residual, out_dtype=out_type)
        assert torch.equal(got, y.to(out_type))


# One and two rows: K below, at and above what the vector unit's kernel takes, its steps of 512 and
# passes of 8 of them ending anywhere, and column counts that end inside a wave's and a workgroup's.
@pytest.mark.parametrize("m", [1, 2])
@pytest.mark.parametrize("n,k", [(1, 513), (3, 520), (8, 1023), (33, 1024), (31, 1025), (50, 1544), (100, 2047), (17, 2048), (9, 2049),
                                 (7, 4096), (1000, 4097), (66, 4103), (5, 9999), (2, 512)])
def test_fused_one_and_two_rows(m, n, k):
    _say("fused one and two rows", m, n, k)
    gen = _gen(n + k)
    a, b, bias = ref.eighths(gen, m, k), ref.eighths(gen, n, k), ref.eighths(gen, n)
    for offset in (0, 1):
        for out_type in (F16, F32):
            residual = ref.eighths(gen, m, n).to(out_type)
            y, z, _, _ = ref.fused(a, b, bias, "relu", residual)
            got, pre = g.gemm_f16_fused_nt(_offset(a, offset), _offset(b, offset), bias, act="relu", residual=residual,
                                           return_pre=True, out_dtype=out_type)
            assert torch.equal(got, y.to(out_type)) and torch.equal(pre, z.to(F16))


# (tile that the automatic choice takes, whether there are more of them than 256 CUs, sizes):
# even, odd and partial K-tile counts, a last row and column of tiles cut short
TILED = [("256x256", False, (3000, 4104, 1024)), ("256x256", False, (3000, 4104, 1032)), ("256x256", True, (6000, 4104, 512)),
         ("256x256", True, (6000, 4104, 1032)), ("256x128", False, (2048, 2056, 512)), ("256x128", False, (2048, 2056, 1032)),
         ("256x128", True, (3000, 4104, 192)), ("256x128", True, (3000, 4104, 200)), ("256x128", True, (4100, 5000, 128)),
         ("128x256", False, (5000, 1000, 384)), ("128x256", False, (4100, 1000, 1032)), ("128x256", True, (4096, 4096, 192)),
         ("128x256", True, (6000, 2056, 200)), ("128x256", True, (6000, 2056, 264)), ("128x128", False, (2100, 1000, 192)),
         ("128x128", False, (2100, 1000, 256)), ("128x128", True, (4100, 1000, 200)), ("128x64", False, (1536, 1000, 192)),
         ("128x64", True, (2048, 2056, 192)), ("64x128", True, (4100, 1000, 192)), ("64x128", True, (2100, 1536, 128)),
         ("64x64", True, (2100, 1000, 128))]


@pytest.mark.parametrize("tile,more,size", TILED)
def test_fused_on_every_tile(tile, more, size):
    _say("fused tiles", tile, more, size)
    m, n, k = size
    names = {v: name[5:] for name, v in vars(g).items() if name.startswith("TILE_")}
    bm, bn = (int(x) for x in tile.split("x"))
    assert names[g.select_tile(m, n, k)] == tile and (-(-m // bm) * -(-n // bn) > 256) == more
    gen = _gen(m + n + k)
    a, b = ref.eighths(gen, m, k), ref.eighths(gen, n, k)
    bias, res = ref.eighths(gen, n), ref.eighths(gen, m, n)
    product = ref.fused(a, b, None, None, None)[1]
    for bias_t in (None, bias, bias.float()):
        for act in (None, "relu"):
            for res_t in (None, res):
                z = product if bias_t is None else product + bias_t.double()
                y = ref.act(act, z) if res_t is None else ref.act(act, z) + res_t.double()
                buf = torch.full((m * n + 64,), 7.0, dtype=F16, device="cuda")
                out = buf[32:32 + m * n].view(m, n)
                got, pre = g.gemm_f16_fused_nt(a, b, bias_t, act=act, residual=res_t, return_pre=True, out=out)
                assert torch.equal(out, y.to(F16)) and torch.equal(pre, z.to(F16)), (bias_t is None, act, res_t is None)
                assert bool((buf[:32] == 7).all()) and bool((buf[32 + m * n:] == 7).all())
                assert torch.equal(g.gemm_f16_fused_nt(a, b, bias_t, act=act, residual=res_t), out)
    y = product + bias.double()
    assert torch.equal(g.gemm_f16_fused_nt(a, b, bias, residual=res.float(), out_dtype=F32), (y + res.double()).float())
    # the other activations, and none of the exact sums' help
    b = ref.normal(gen, n, k, std=2 * k**-0.5)
    for act in ("gelu", "gelu_tanh", "silu"):
        y, z, err, ez = ref.fused(a, b, bias, act, None)
        assert ref.worst(g.gemm_f16_fused_nt(a, b, bias, act=act), y, err, F16) <= 1


# Rows that are not 16-byte aligned, on each of their tiles and in parts of K: whole dwords (K even,
# operands at an even element) and not; the K loop's first, last and only K-tiles broken.
@pytest.mark.parametrize("m,n,k", [(3000, 4104, 1022), (3000, 4104, 1023), (5000, 1000, 391), (2100, 1000, 193), (2048, 2056, 1030),
                                   (128, 512, 4099), (128, 512, 4098), (300, 264, 77), (257, 100, 66), (70, 70, 1), (4352, 64, 2051),
                                   (1500, 300, 129), (1025, 1032, 2047)])
def test_fused_rows_of_any_alignment(m, n, k):
    _say("fused unaligned rows", m, n, k)
    gen = _gen(m + n + k)
    a, b, bias = ref.eighths(gen, m, k), ref.eighths(gen, n, k), ref.eighths(gen, n)
    res = ref.eighths(gen, m, n)
    y, z, _, _ = ref.fused(a, b, bias, "relu", res)
    for by_a, by_b in ((0, 0), (2, 0), (0, 1), (1, 3)):
        got, pre = g.gemm_f16_fused_nt(_offset(a, by_a), _offset(b, by_b), bias, act="relu", residual=res, return_pre=True)
        assert torch.equal(got, y.to(F16)) and torch.equal(pre, z.to(F16)), (by_a, by_b)
    assert torch.equal(g.gemm_f16_fused_nt(a, b, bias, act="relu", residual=res.float(), out_dtype=F32), y.float())


# Every number of columns left over, every path; results at each offset of their element; in place too.
@pytest.mark.parametrize("n", range(257, 264))
@pytest.mark.parametrize("m,k", [(1, 1024), (13, 256), (200, 512), (70, 4096), (4352, 64)])
def test_fused_columns_left_over(m, n, k):
    _say("fused columns left over", m, n, k)
    gen = _gen(m + n + k)
    a, b, bias = ref.eighths(gen, m, k), ref.eighths(gen, n, k), ref.eighths(gen, n)
    for out_type in (F16, F32):
        res = ref.eighths(gen, m, n).to(out_type)
        y, z, _, _ = ref.fused(a, b, bias, "relu", res)
        buf = torch.full((m * n + 64,), 7.0, dtype=out_type, device="cuda")
        for by in (16, 17, 18):
            out = buf[by:by + m * n].view(m, n).copy_(res)
            got, pre = g.gemm_f16_fused_nt(a, b, bias, act="relu", residual=out, return_pre=True, out=out, out_dtype=out_type)
            assert torch.equal(out, y.to(out_type)) and torch.equal(pre, z.to(F16)), (out_type, by)
            assert bool((buf[:by] == 7).all()) and bool((buf[by + m * n:] == 7).all())
            buf.fill_(7.0)


# Rows of C of fewer columns than a chunk, on every way there is: one and two rows, few rows, tiles, the
# ring, parts of K, unaligned rows.
@pytest.mark.parametrize("n", range(1, 9))
@pytest.mark.parametrize("m,k", [(1, 2048), (2, 64), (5, 300), (20, 4096), (70, 100), (300, 4096), (300, 4097), (6000, 128), (5000, 4096)])
def test_fused_fewer_columns_than_a_chunk(m, n, k):
    _say("fused fewer columns", m, n, k)
    gen = _gen(m + n + k)
    a, b, bias = ref.eighths(gen, m, k), ref.eighths(gen, n, k), ref.eighths(gen, n)
    for out_type in (F16, F32):
        res = ref.eighths(gen, m, n).to(out_type)
        y, z, _, _ = ref.fused(a, b, bias, "relu", res)
        buf = torch.full((m * n + 64,), 7.0, dtype=out_type, device="cuda")
        out = buf[17:17 + m * n].view(m, n).copy_(res)
        got, pre = g.gemm_f16_fused_nt(a, b, bias, act="relu", residual=out, return_pre=True, out=out, out_dtype=out_type)
        assert torch.equal(out, y.to(out_type)) and torch.equal(pre, z.to(F16)), out_type
        assert bool((buf[:17] == 7).all()) and bool((buf[17 + m * n:] == 7).all())


@pytest.mark.parametrize("m,n,k", [(1, 1000, 2048), (33, 200, 777), (200, 264, 512), (1500, 1200, 320), (4352, 4096, 256)])
@pytest.mark.parametrize("act", ref.ACTS)
def test_fused_random(m, n, k, act):
    _say("fused random", m, n, k, act)
    gen = _gen(m * n + k)
    a, b = ref.normal(gen, m, k), ref.normal(gen, n, k, std=2 * k**-0.5)
    bias = torch.randn(n, generator=gen, device="cuda")
    for out_type in (F16, F32):
        residual = torch.randn(m, n, generator=gen, device="cuda").to(out_type)
        y, z, err, ez = ref.fused(a, b, bias, act, residual)
        got, pre = g.gemm_f16_fused_nt(a, b, bias, act=act, residual=residual, return_pre=True, out_dtype=out_type)
        assert ref.worst(got, y, err, out_type) <= 1
        assert ref.worst(pre, z, ez, F16) <= 1
        assert torch.equal(got, g.gemm_f16_fused_nt(a, b, bias, act=act, residual=residual, out_dtype=out_type))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_activations_over_their_whole_range(act):
    """z itself through the epilogue (a one times z): every finite fp16 value, in fp32."""
    z = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.float16).cuda()
    z = z[torch.isfinite(z)]
    a = torch.zeros(len(z), 8, dtype=F16, device="cuda")
    a[:, 0] = z
    b = torch.zeros(8, 8, dtype=F16, device="cuda")
    b[:, 0] = 1
    got = g.gemm_f16_fused_nt(a, b, act=act, out_dtype=F32)
    want = ref.act(act, z.double())
    # the hardware's exp2 and rcp give 0 for results below 2^-126, the smallest normal number:
    # a sigmoid below that is 0, and times |z| < 90 (where it gets there) off by 90 2^-126 < 2^-119
    err = ref.act_error(act, z.double()) * want.abs() + 2.0**-119
    assert ref.worst(got, want[:, None].expand(-1, 8), err[:, None].expand(-1, 8), F32) <= 1
    pre = z.clone()[:, None].expand(-1, 8).contiguous()
    dz, dbias = g.gemm_f16_fused_grad(torch.ones_like(pre), pre, act=act)
    w_dz, w_db, e_dz, e_db = ref.fused_grad(torch.ones_like(pre), pre, act)
    assert ref.worst(dz, w_dz, e_dz, F16) <= 1 and ref.worst(dbias, w_db, e_db, F32) <= 1


@pytest.mark.parametrize("m", [2, 200])
def test_fused_what_is_not_finite(m):
    """An infinity or NaN of a row or column stays there, and gives what the formulas give."""
    gen = _gen(5)
    a, b = ref.normal(gen, m, 64), ref.normal(gen, 72, 64, std=0.125)
    a[0, 3], b[5, 9], a[1, 7] = INF, NAN, 60000.0
    b[7, 7] = 60000.0
    for act in ref.ACTS:
        z = a.double() @ b.double().T
        want = ref.act(act, z)
        got = g.gemm_f16_fused_nt(a, b, act=act, out_dtype=F32)
        clean = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), clean)
        assert bool(torch.isnan(got[:, 5]).all()) and bool((got[0][z[0] == INF] == INF).all())
        assert torch.allclose(got[clean].double(), want[clean], rtol=1e-4, atol=1e-4)
        assert float(got[1, 7]) == pytest.approx(3.6e9, rel=1e-3)
        # past fp16's range the rounded result is an infinity
        assert float(g.gemm_f16_fused_nt(a, b, act=act)[1, 7]) == INF


@pytest.mark.parametrize("what", ["a", "b", "bias", "residual", "out", "n"])
@pytest.mark.parametrize("m,n,k", [(5, 64, 128), (150, 136, 192)])
def test_fused_any_alignment(what, m, n, k):
    _say("fused alignment", what, m, n, k)
    gen = _gen(k)
    n = n + 3 if what == "n" else n
    t = {"a": ref.eighths(gen, m, k), "b": ref.eighths(gen, n, k), "bias": ref.eighths(gen, n), "residual": ref.eighths(gen, m, n)}
    y = ref.fused(t["a"], t["b"], t["bias"], None, t["residual"])[0]
    buf = torch.full((m * n + 33,), 7.0, dtype=F16, device="cuda")
    start = 1 if what == "out" else 16
    out = buf[start:start + m * n].view(m, n)
    if what in t:
        t[what] = _offset(t[what], 1)
    got = g.gemm_f16_fused_nt(t["a"], t["b"], t["bias"], residual=t["residual"], out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, y.to(F16))
    assert bool((buf[:start] == 7).all()) and bool((buf[start + m * n:] == 7).all())


@pytest.mark.parametrize("m,n,k", [(7, 264, 512), (40, 100, 333), (300, 264, 512), (2200, 2100, 136), (4352, 4096, 256)])
@pytest.mark.parametrize("out_type", [F16, F32])
def test_fused_onto_the_residual(m, n, k, out_type):
    _say("fused in place", m, n, k, out_type)
    gen = _gen(n)
    a, b, x = ref.eighths(gen, m, k), ref.eighths(gen, n, k), ref.eighths(gen, m, n).to(out_type)
    y = ref.fused(a, b, None, "relu", x)[0]
    got = g.gemm_f16_fused_nt(a, b, act="relu", residual=x, out_dtype=out_type, out=x)
    assert got is x and torch.equal(x, y.to(out_type))


def test_fused_without_k_or_rows():
    gen = _gen(1)
    a, b = torch.zeros(70, 0, dtype=F16, device="cuda"), torch.zeros(33, 0, dtype=F16, device="cuda")
    bias, residual = torch.randn(33, generator=gen, device="cuda"), ref.normal(gen, 70, 33)
    got, pre = g.gemm_f16_fused_nt(a, b, bias, act="silu", residual=residual, return_pre=True)
    y, z, err, ez = ref.fused(a, b, bias, "silu", residual)
    assert ref.worst(got, y, err, F16) <= 1 and torch.equal(pre, bias.half().expand(70, 33))
    assert torch.equal(g.gemm_f16_fused_nt(a, b), torch.zeros(70, 33, dtype=F16, device="cuda"))
    assert g.gemm_f16_fused_nt(a[:0], b).shape == (0, 33)
    assert g.gemm_f16_fused_nt(a, b[:0]).shape == (70, 0)


def test_fused_outputs_past_2_31_elements():
    m, n = 600_000, 4096
    gen = _gen(2)
    a, b = ref.eighths(gen, m, 8), ref.eighths(gen, n, 8)
    bias = ref.eighths(gen, n)
    got = g.gemm_f16_fused_nt(a, b, bias, act="relu")
    rows = torch.tensor([0, 1, 255, 524_287, 524_288, 524_289, m - 257, m - 1], device="cuda")
    want = ref.fused(a[rows], b, bias, "relu", None)[0].to(F16)
    assert torch.equal(got[rows], want)


@pytest.mark.parametrize("m,n", [(1, 1), (1, 4096), (5, 7), (33, 40), (1000, 24), (777, 130), (4096, 264), (5000, 1003), (20000, 64),
                                 *((300, n) for n in range(2, 17))])
@pytest.mark.parametrize("act", ref.ACTS)
def test_fused_grad(m, n, act):
    _say("fused grad", m, n, act)
    gen = _gen(m + n)
    for dy_type in (F16, F32):
        dy = torch.randn(m, n, generator=gen, device="cuda").to(dy_type)
        pre = ref.normal(gen, m, n, std=2.0) if act else None
        w_dz, w_db, e_dz, e_db = ref.fused_grad(dy, pre, act)
        dz, dbias = g.gemm_f16_fused_grad(dy, pre, act=act)
        if act:
            assert dz.dtype == F16 and ref.worst(dz, w_dz, e_dz, F16) <= 1
        else:
            assert dz is dy
        assert ref.worst(dbias, w_db, e_db, F32) <= 1
        again = g.gemm_f16_fused_grad(dy, pre, act=act)
        assert torch.equal(again[1], dbias) and torch.equal(again[0], dz)
        alone, none = g.gemm_f16_fused_grad(dy, pre, act=act, bias_grad=False)
        assert none is None and torch.equal(alone, dz)


def test_fused_grad_in_place_unaligned_and_empty():
    gen = _gen(3)
    dy, pre = ref.normal(gen, 300, 72), ref.normal(gen, 300, 72)
    want = g.gemm_f16_fused_grad(dy, pre, act="silu")
    off = g.gemm_f16_fused_grad(_offset(dy, 1), _offset(pre, 3), act="silu")
    assert torch.equal(off[0], want[0])
    assert torch.allclose(off[1], want[1], rtol=1e-5, atol=1e-4)
    own = dy.clone()
    rc = g.lib().gemm_f16_fused_grad(300, 72, own.data_ptr(), 0, pre.data_ptr(), 4, own.data_ptr(), None, None, 0,
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == g.OK and torch.equal(own, want[0])
    dz, dbias = g.gemm_f16_fused_grad(dy[:0], pre[:0], act="gelu")
    assert dz.shape == (0, 72) and torch.equal(dbias, torch.zeros(72, device="cuda"))


@pytest.mark.parametrize("m,n", [(40, 9), (300, 75), (1000, 131), (70, 263)])
@pytest.mark.parametrize("act", ["relu", "silu"])
def test_fused_grad_in_place_with_columns_left_over(m, n, act):
    """The last columns are read with the ones before them, which another thread overwrites, and where
    something may not be finite."""
    gen = _gen(m + n)
    dy, pre = ref.normal(gen, m, n), ref.normal(gen, m, n)
    dy[0, n - 8], dy[m - 1, n - 9] = INF, NAN
    want, dbias = g.gemm_f16_fused_grad(dy, pre, act=act)
    bad = ~torch.isfinite(dbias)
    assert bool(bad[n - 9]) == (act != "relu" or float(pre[m - 1, n - 9]) > 0)  # (relu's slope is a choice, not a factor)
    assert not bool(bad[:n - 9].any()) and not bool(bad[n - 7:].any())
    own = dy.clone()
    rc = g.lib().gemm_f16_fused_grad(m, n, own.data_ptr(), 0, pre.data_ptr(), {"relu": 1, "silu": 4}[act], own.data_ptr(), None,
                                     None, 0, torch.cuda.current_stream().cuda_stream)
    assert rc == g.OK and torch.equal(own.view(torch.int16), want.view(torch.int16))


def test_fused_grad_past_2_31_elements():
    m, n = 540_000, 4096
    dy = torch.ones(m, n, dtype=F16, device="cuda")
    pre = torch.ones(m, n, dtype=F16, device="cuda")
    pre[m - 1] = -1.0
    dz, dbias = g.gemm_f16_fused_grad(dy, pre, act="relu")
    assert bool((dz[m - 1] == 0).all()) and bool((dz[m - 2] == 1).all()) and bool((dbias == m - 1).all())


# ---- routing ------------------------------------------------------------------------

def _check_route(logits, fan, **how):
    ids, gates = g.route(logits, fan, **how)
    torch.cuda.synchronize()
    w_ids, w_gates = ref.route(logits, fan, **how)
    assert torch.equal(ids.cpu().long(), w_ids)
    # exp, with its argument's rounding (differences of logits up to 100), the sum's terms, a quotient and the scale
    terms = logits.shape[1] if how.get("score", "softmax") == "softmax" and not how.get("renormalize", True) else fan
    # (a gate below fp32's normal numbers, 2^-126, may be 0: exp(-200) is 1.4e-87)
    err = (100 + terms + 12) * 2 * ref.U * w_gates.abs() + 2.0**-126
    assert ref.worst(gates.cpu(), w_gates, err, F32) <= 1
    again = g.route(logits, fan, **how)
    assert torch.equal(ids, again[0]) and torch.equal(gates, again[1])
    return ids, gates


@pytest.mark.parametrize("tokens,experts,fan", [(1, 1, 1), (1, 8, 2), (64, 8, 2), (3, 16, 16), (17, 20, 3), (130, 64, 6), (65, 100, 8),
                                                (40, 128, 32), (50, 160, 17), (33, 256, 8), (20, 257, 8), (12, 384, 6), (9, 600, 32),
                                                (6, 1024, 8), (5, 1500, 10), (3, 2048, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(tokens, experts, fan, score):
    _say("route", tokens, experts, fan, score)
    gen = _gen(tokens * experts + fan)
    for dtype in (F16, F32):
        logits = (torch.randn(tokens, experts, generator=gen, device="cuda") * 2).to(dtype)
        bias = torch.randn(experts, generator=gen, device="cuda") * 0.1
        for b in (None, bias):
            for renormalize in (True, False):
                _check_route(logits, fan, score=score, bias=b, renormalize=renormalize, scale=1.0 if renormalize else 2.5)


@pytest.mark.parametrize("experts,groups,top_groups,fan", [(8, 2, 1, 2), (64, 8, 3, 6), (256, 8, 4, 8), (160, 8, 3, 6), (60, 20, 7, 9),
                                                           (64, 64, 5, 5), (512, 16, 2, 12), (2048, 64, 9, 32), (40, 8, 8, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_in_groups(experts, groups, top_groups, fan, group_top):
    _say("route groups", experts, groups, top_groups, fan, group_top)
    gen = _gen(experts + groups)
    logits = torch.randn(37, experts, generator=gen, device="cuda") * 2
    bias = torch.randn(experts, generator=gen, device="cuda") * 0.2
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            _check_route(logits, fan, score=score, bias=b, groups=groups, top_groups=top_groups, group_top=group_top, scale=2.5)
            _check_route(logits.half(), fan, score=score, bias=b, groups=groups, top_groups=top_groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masked_and_infinite(score, groups):
    """Experts without a finite key, rows with too few or none, infinities, ties, padding."""
    gen = _gen(7)
    logits = torch.randn(41, 16, generator=gen, device="cuda") * 3
    logits[0] = -INF
    logits[1, 1:] = -INF
    logits[2, ::2] = -INF
    logits[3] = NAN
    logits[4, 5] = NAN
    logits[5, [2, 9]] = INF
    logits[6] = INF
    logits[7] = 0.5
    logits[8, :8] = torch.finfo(F32).min
    logits[9] = torch.finfo(F32).min
    logits[10] = torch.finfo(F32).max
    logits[11, 3:] = -200.0
    logits[12, :12] = -INF
    logits[13:20] = torch.randint(-2, 3, (7, 16), generator=gen, device="cuda").float()  # ties
    bias = torch.randn(16, generator=gen, device="cuda")
    odd = bias.clone()
    odd[3], odd[8], odd[11] = -INF, NAN, INF
    for b in (None, torch.zeros(16, device="cuda"), bias, odd):
        for renormalize in (True, False):
            for group_top in (1, 2):
                how = dict(score=score, bias=b, groups=groups, top_groups=2 if groups > 1 else 1, group_top=group_top, renormalize=renormalize)
                ids, gates = _check_route(logits, 4, **how)
                assert ids[0].tolist() == [-1] * 4 and gates[0].tolist() == [0.0] * 4
                order, inverse, offsets = g.group_rows(ids, 16)
                assert int(offsets[-1]) == int((ids >= 0).sum())


def test_route_tells_close_keys_apart():
    """Keys that agree in fp32, or come out in the wrong order there, and differ in 64 bits."""
    base = torch.linspace(-1, 1, 16).repeat(64, 1)
    # sigmoids that are all 1 in fp32: the larger logit wins, wherever it is
    logits = base.clone()
    for t in range(64):
        logits[t, t % 16], logits[t, (t + 5) % 16], logits[t, (t + 9) % 16] = 20.0, 22.0, 21.0
    _check_route(logits.cuda(), 2, score="sigmoid", bias=torch.zeros(16, device="cuda"))
    # scores and biases whose sums differ by parts of an fp32 step
    gen = torch.Generator().manual_seed(3)
    l = torch.randn(512, 16, generator=gen)
    for score in ("softmax", "sigmoid"):
        s = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
        bias = (0.5 - s[0]).float()  # token 0: all keys 1/2 within a rounding
        for groups in (1, 4):
            _check_route(l[:1].cuda().repeat(5, 1), 4, score=score, bias=bias.cuda(), groups=groups, top_groups=2 if groups > 1 else 1,
                         group_top=2)
    # exact ties in 64 bits go to the lowest index
    tied = torch.full((9, 64), 1.25).cuda()
    ids, _ = _check_route(tied, 6, score="sigmoid", bias=torch.full((64,), 0.1, device="cuda"), groups=8, top_groups=3, group_top=2)
    assert ids.tolist() == [[0, 1, 2, 3, 4, 5]] * 9


@pytest.mark.parametrize("experts,groups,fan", [(256, 8, 8), (64, 16, 6), (40, 8, 5), (16, 4, 4), (16, 16, 3), (100, 20, 8), (8, 2, 2),
                                                (512, 8, 8)])
@pytest.mark.parametrize("alike", ["groups", "experts"])
def test_route_tells_close_groups_apart(experts, groups, fan, alike):
    """Groups whose values differ by steps of a logit in fp32: each a copy of the same logits but for those
    steps; or all experts alike but for them."""
    _say("route close groups", experts, groups, fan, alike)
    gen = _gen(experts + groups)
    per = experts // groups
    base = torch.randn(33, 1, per, generator=gen, device="cuda") if alike == "groups" else torch.full((33, 1, per), 0.75, device="cuda")
    steps = torch.randint(-2, 3, (33, groups, per), generator=gen, device="cuda")
    logits = (base.expand(-1, groups, -1) * (1 + steps * 2.0**-23)).reshape(33, experts)
    logits[::5, ::3] = -INF
    tilt = torch.randn(1, per, generator=gen, device="cuda").mul_(0.1).expand(groups, -1).reshape(-1).contiguous()
    for bias in (None, tilt):
        for group_top in (1, 2):
            _check_route(logits, fan, score="sigmoid", bias=bias, groups=groups, top_groups=max(1, groups // 2), group_top=group_top)


def test_route_unaligned_logits_and_no_tokens():
    gen = _gen(4)
    logits = torch.randn(30, 64, generator=gen, device="cuda")
    want = _check_route(logits, 4)
    for dtype, by in ((F32, 1), (F16, 1), (F16, 3)):
        at = _offset(logits.to(dtype), by)
        got = g.route(at, 4)
        same = g.route(logits.to(dtype), 4)
        assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
    assert want[0].shape == (30, 4)
    ids, gates = g.route(logits[:0], 4)
    assert ids.shape == gates.shape == (0, 4)
    with pytest.raises(g.GemmError):
        g.route(logits, 65)
    with pytest.raises(g.GemmError):
        g.route(logits, 4, groups=5)


@pytest.mark.parametrize("tokens,experts,fan", [(1, 1, 1), (5, 8, 2), (64, 16, 16), (33, 60, 5), (100, 256, 8), (7, 128, 32), (9, 300, 20),
                                                (4, 1024, 8), (3, 2048, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad(tokens, experts, fan, score, renormalize):
    _say("route grad", tokens, experts, fan, score, renormalize)
    gen = _gen(experts + fan)
    for dtype in (F16, F32):
        logits = (torch.randn(tokens, experts, generator=gen, device="cuda") * 2).to(dtype)
        how = dict(score=score, renormalize=renormalize, scale=1.5)
        ids, _ = g.route(logits, fan, **how)
        dg = torch.randn(tokens, fan, generator=gen, device="cuda")
        leaf = logits.double().requires_grad_()
        gates = ref.gates_of(leaf, ids.long(), **how)
        want, = torch.autograd.grad(gates, leaf, dg.double())
        got = g.route_grad(logits, ids, dg, **how)
        assert got.dtype == dtype
        # terms c and the weighted sum of c, each of up to fan products, times a score: the
        # roundings of the gates (as in _check_route) on the sum of magnitudes
        with torch.no_grad():
            s = torch.softmax(leaf, 1) if score == "softmax" else torch.sigmoid(leaf) * torch.sigmoid(-leaf)
            c = 1.5 * dg.double().abs()
            picked = torch.zeros_like(leaf).scatter_(1, ids.long(), c)
            if renormalize:
                p = (torch.softmax(leaf, 1) if score == "softmax" else torch.sigmoid(leaf)).gather(1, ids.long())
                share = p / p.sum(1, keepdim=True)
                tail = 1.0 if score == "softmax" else torch.sigmoid(-leaf).gather(1, ids.long())
                mag = torch.zeros_like(leaf).scatter_(1, ids.long(), share * tail * (c + (c * share).sum(1, keepdim=True)))
            elif score == "softmax":
                mag = s * (picked + (c * s.gather(1, ids.long())).sum(1, keepdim=True))
            else:
                mag = s * picked
        err = (40 + 2 * max(fan, experts if score == "softmax" and not renormalize else 0) + 16) * 2 * ref.U * mag
        # (where the terms cancel, the oracle's own sums of up to 2048 of them, below 2^4, in 64 bits)
        assert ref.worst(got, want, err + 2.0**-38, dtype) <= 1
        assert torch.equal(got, g.route_grad(logits, ids, dg, **how))


def test_route_grad_against_differences():
    gen = _gen(9)
    logits = torch.randn(6, 12, generator=gen, device="cuda")
    dg = torch.randn(6, 3, generator=gen, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            ids, _ = g.route(logits, 3, score=score, renormalize=renormalize)
            got = g.route_grad(logits, ids, dg, score=score, renormalize=renormalize).double()
            x = logits.double()
            for t, e in ((0, 0), (1, int(ids[1, 0])), (2, int(ids[2, 2])), (5, 11)):
                moved = []
                for step in (1e-5, -1e-5):
                    u = x.clone()
                    u[t, e] += step
                    moved.append((ref.gates_of(u, ids.long(), score, renormalize, 1.0) * dg.double()).sum())
                assert abs(float((moved[0] - moved[1]) / 2e-5 - got[t, e])) < 1e-5


def test_route_grad_of_masked_rows():
    """No chosen expert, ids of none, logits of -inf: zeros there, and finite everywhere."""
    gen = _gen(11)
    logits = torch.randn(8, 16, generator=gen, device="cuda")
    logits[0] = -INF
    logits[1, 2:] = -INF
    logits[2, ::3] = NAN
    logits[3] = -300.0  # sigmoids that are 0 in fp32
    dg = torch.randn(8, 4, generator=gen, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            ids, gates = g.route(logits, 4, score=score, renormalize=renormalize)
            ids[7, 1], ids[7, 2] = 99, -5
            d = g.route_grad(logits, ids, dg, score=score, renormalize=renormalize)
            assert bool(torch.isfinite(d).all()) and bool(torch.isfinite(gates).all())
            assert bool((d[0] == 0).all()) and bool((d[1, 2:] == 0).all()) and bool((d[2, ::3] == 0).all())
            keep = torch.zeros(16, dtype=torch.bool, device="cuda")
            keep[ids[7][[0, 3]].long()] = True
            if renormalize or score == "sigmoid":
                assert bool((d[7][~keep] == 0).all()) and bool((d[7][keep] != 0).all())
    # the same expert twice: both gates' gradients
    twice = torch.tensor([[3, 3]], dtype=torch.int32, device="cuda")
    d = g.route_grad(logits[4:5], twice, dg[4:5, :2].contiguous(), renormalize=False)
    leaf = logits[4:5].double().requires_grad_()
    want, = torch.autograd.grad(torch.softmax(leaf, 1).gather(1, twice.long()), leaf, dg[4:5, :2].double())
    assert torch.allclose(d.double(), want, atol=1e-6)


# ---- the way back ---------------------------------------------------------------------

def _routed(gen, tokens, fan, experts, dropped=0.1):
    ids = torch.rand(tokens, experts, generator=gen, device="cuda").argsort(1)[:, :fan].to(torch.int32)
    ids = torch.where(torch.rand(tokens, fan, generator=gen, device="cuda") < dropped, -1, ids).to(torch.int32)
    return g.group_rows(ids, experts)


COMBINE = [(1, 1, 1), (1, 2, 4096), (5, 1, 7), (33, 2, 64), (40, 3, 100), (100, 8, 520), (17, 11, 40), (300, 4, 1032), (64, 2, 3001), (9, 32, 8),
           (3, 8, 7000), (40, 3, 9001), (700, 6, 4100)]


@pytest.mark.parametrize("tokens,fan,n", COMBINE)
def test_combine(tokens, fan, n):
    _say("combine", tokens, fan, n)
    gen = _gen(tokens + fan + n)
    experts = max(fan, 4)
    _, inverse, offsets = _routed(gen, tokens, fan, experts)
    last = int(offsets[-1])
    for rows_type in (F16, F32):
        rows = torch.randn(tokens * fan, n, generator=gen, device="cuda").to(rows_type)
        rows[last:] = NAN  # what belongs to no expert is not looked at
        gates = torch.rand(tokens, fan, generator=gen, device="cuda")
        for out_type in (F16, F32):
            for w, with_residual in ((gates, True), (gates, False), (None, False)):
                residual = torch.randn(tokens, n, generator=gen, device="cuda").to(out_type) if with_residual else None
                y, err = ref.combine(rows, inverse, last, fan, w, residual)
                got = g.combine_rows(rows, inverse, offsets, fan, gates=w, residual=residual, out_dtype=out_type)
                assert ref.worst(got, y, err, out_type) <= 1
                if with_residual:
                    own = residual.clone()
                    assert g.combine_rows(rows, inverse, offsets, fan, gates=w, residual=own, out_dtype=out_type, out=own) is own
                    assert torch.equal(own, got)


@pytest.mark.parametrize("tokens,fan,n", COMBINE)
def test_combine_grad(tokens, fan, n):
    _say("combine grad", tokens, fan, n)
    gen = _gen(tokens + fan + n)
    _, inverse, offsets = _routed(gen, tokens, fan, max(fan, 4))
    last = int(offsets[-1])
    for rows_type, dy_type, drows_type in ((F16, F16, F16), (F32, F16, F16), (F16, F32, F32)):
        rows = torch.randn(tokens * fan, n, generator=gen, device="cuda").to(rows_type)
        rows[last:] = NAN
        gates = torch.rand(tokens, fan, generator=gen, device="cuda")
        gates[0, 0] = 0.0
        dy = torch.randn(tokens, n, generator=gen, device="cuda").to(dy_type)
        w_rows, w_gates, e_rows, e_gates = ref.combine_grad(dy, rows, inverse, last, gates)
        drows, dgates = g.combine_rows_grad(dy, rows, inverse, offsets, gates, rows_dtype=drows_type)
        assert drows.dtype == drows_type
        assert ref.worst(drows, w_rows, e_rows, drows_type) <= 1 and ref.worst(dgates, w_gates, e_gates, F32) <= 1
        again = g.combine_rows_grad(dy, rows, inverse, offsets, gates, rows_dtype=drows_type)
        assert torch.equal(again[0], drows) and torch.equal(again[1], dgates)


def test_combine_unaligned_empty_and_all_dropped():
    gen = _gen(6)
    _, inverse, offsets = _routed(gen, 50, 2, 4)
    rows, gates = ref.normal(gen, 100, 72), torch.rand(50, 2, generator=gen, device="cuda")
    residual, dy = ref.normal(gen, 50, 72), ref.normal(gen, 50, 72)
    want = g.combine_rows(rows, inverse, offsets, 2, gates=gates, residual=residual)
    got = g.combine_rows(_offset(rows, 1), inverse, offsets, 2, gates=gates, residual=_offset(residual, 1), out=_offset(residual, 5))
    assert torch.equal(got, want)
    w_rows, w_gates = g.combine_rows_grad(dy, rows, inverse, offsets, gates)
    d_rows, d_gates = g.combine_rows_grad(_offset(dy, 1), _offset(rows, 3), inverse, offsets, gates)
    assert torch.equal(d_rows, w_rows) and torch.allclose(d_gates, w_gates, rtol=1e-5, atol=1e-4)
    _, inverse, offsets = g.group_rows(torch.full((50, 2), -1, dtype=torch.int32, device="cuda"), 4)
    assert torch.equal(g.combine_rows(rows, inverse, offsets, 2, gates=gates, residual=residual), residual)
    d_rows, d_gates = g.combine_rows_grad(dy, rows, inverse, offsets, gates)
    assert not bool(d_rows.any()) and not bool(d_gates.any())
    assert g.combine_rows(rows[:0], inverse[:0], offsets, 2, gates=gates[:0]).shape == (0, 72)


def test_combine_bad_places_touch_nothing_else():
    """Places out of range add nothing; rows that no place names keep what they hold."""
    gen = _gen(8)
    rows, dy = ref.normal(gen, 8, 40), ref.normal(gen, 4, 40)
    gates = torch.ones(4, 2, device="cuda")
    inverse = torch.tensor([0, -1, 1, 8, 2, 2**31 - 1, 3, -(2**31)], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 2**31 - 1], dtype=torch.int32, device="cuda")
    assert torch.equal(g.combine_rows(rows, inverse, offsets, 2, gates=gates), rows[:4])
    drows = torch.full((8, 40), 7.0, dtype=F16, device="cuda")
    dgates = torch.empty(4, 2, device="cuda")
    rc = g.lib().gemm_f16_combine_rows_grad(4, 2, 40, 1, dy.data_ptr(), 0, rows.data_ptr(), 0, inverse.data_ptr(), offsets.data_ptr(),
                                            gates.data_ptr(), drows.data_ptr(), 0, dgates.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == g.OK and torch.equal(drows[:4], dy) and bool((drows[4:] == 7).all())
    assert bool((dgates[:, 1] == 0).all()) and torch.allclose(dgates[:, 0], (dy.double() * rows[:4].double()).sum(1).float(), atol=1e-4)


def test_combine_rows_past_2_31_elements():
    tokens, fan, n = 270_000, 2, 4096
    ids = torch.zeros(tokens, fan, dtype=torch.int32, device="cuda")
    ids[:, 1] = 1
    _, inverse, offsets = g.group_rows(ids, 2)
    rows = torch.empty(tokens * fan, n, dtype=F16, device="cuda")
    rows[:tokens] = 1.0
    rows[tokens:] = 2.0
    rows[-1] = 5.0
    gates = torch.full((tokens, fan), 0.5, device="cuda")
    y = g.combine_rows(rows, inverse, offsets, fan, gates=gates)
    assert bool((y[:-1] == 1.5).all()) and bool((y[-1] == 3.0).all())
    drows, dgates = g.combine_rows_grad(y, rows, inverse, offsets, gates)
    assert bool((drows[-1] == 1.5).all()) and bool((drows[tokens:-1] == 0.75).all())
    assert dgates[-1].tolist() == [3.0 * n, 15.0 * n]


# ---- together ---------------------------------------------------------------------------

def _layer(gen, tokens, width, hidden, experts):
    n = ref.normal
    return {"x": n(gen, tokens, width), "router": n(gen, experts, width, std=width**-0.5), "bias": torch.randn(experts, generator=gen, device="cuda") * 0.01,
            "w": n(gen, experts, width, width, std=width**-0.5), "up": n(gen, hidden, width, std=width**-0.5),
            "b_up": torch.randn(hidden, generator=gen, device="cuda") * 0.1, "down": n(gen, width, hidden, std=hidden**-0.5), "one": torch.tensor([0, tokens], dtype=torch.int32, device="cuda")}


def _forward(t, fan):
    """x + shared feed-forward(x) + routed experts(x), and what its backward pass takes."""
    logits = g.gemm_f16_fused_nt(t["x"], t["router"], out_dtype=F32)
    ids, gates = g.route(logits, fan, score="sigmoid", bias=t["bias"], groups=2, top_groups=1, group_top=2)
    order, inverse, offsets = g.group_rows(ids, len(t["w"]))
    rows = g.gemm_f16_grouped_nt(t["x"], t["w"], offsets, index=order, fan=fan)
    hidden, pre = g.gemm_f16_fused_nt(t["x"], t["up"], t["b_up"], act="gelu_tanh", return_pre=True)
    shared = g.gemm_f16_fused_nt(hidden, t["down"], residual=t["x"], out_dtype=F16)
    y = g.combine_rows(rows, inverse, offsets, fan, gates=gates, residual=shared)
    return y, (logits, ids, gates, order, inverse, offsets, rows, hidden, pre)


def _backward(t, fan, dy, kept):
    logits, ids, gates, order, inverse, offsets, rows, hidden, pre = kept
    one = t["one"]  # all tokens in one segment
    drows, dgates = g.combine_rows_grad(dy, rows, inverse, offsets, gates)
    dlogits = g.route_grad(logits, ids, dgates, score="sigmoid")
    d16 = dy.half()
    dx = dy + g.combine_rows(g.gemm_f16_grouped_nn(drows, t["w"], offsets, out_dtype=F32), inverse, offsets, fan, out_dtype=F32)
    token = torch.div(order, fan, rounding_mode="floor").long()
    grads = {"w": g.gemm_f16_grouped_tn(drows, t["x"][token], offsets, out_dtype=F32)}
    grads["down"] = g.gemm_f16_grouped_tn(d16, hidden, one, out_dtype=F32)[0]
    dz, grads["b_up"] = g.gemm_f16_fused_grad(g.gemm_f16_nn_f32(d16, t["down"]), pre, act="gelu_tanh")
    grads["up"] = g.gemm_f16_grouped_tn(dz, t["x"], one, out_dtype=F32)[0]
    dl = dlogits.half()
    grads["router"] = g.gemm_f16_grouped_tn(dl, t["x"], one, out_dtype=F32)[0]
    grads["x"] = dx + g.gemm_f16_nn_f32(dz, t["up"]) + g.gemm_f16_nn_f32(dl, t["router"])
    return grads


def test_a_routed_layer_with_its_gradients():
    """Against the whole layer in 64 bits, the choice of experts held fixed.  The chain rounds
    to fp16 five times between the layer's ends (2^-11 each); 2% of the largest value bounds
    what that and the sums make of it with room, and a wrong factor or row does not pass."""
    tokens, width, experts, fan = 200, 256, 8, 2
    gen = _gen(21)
    t = _layer(gen, tokens, width, 512, experts)
    y, kept = _forward(t, fan)
    leaves = {k: v.double().requires_grad_() for k, v in t.items() if k not in ("bias", "one")}
    x, ids = leaves["x"], kept[1].long()
    gates = ref.gates_of(x @ leaves["router"].T, ids, "sigmoid", True, 1.0)
    want = x + ref.act("gelu_tanh", x @ leaves["up"].T + leaves["b_up"]) @ leaves["down"].T
    for f in range(fan):
        each = torch.stack([x[i] @ leaves["w"][ids[i, f]].T for i in range(tokens)])
        want = want + gates[:, f, None] * each
    assert float((y.double() - want.detach()).abs().max()) < 0.02 * float(want.detach().abs().max())
    w_ids, _ = ref.route(kept[0], fan, score="sigmoid", bias=t["bias"], groups=2, top_groups=1, group_top=2)
    assert torch.equal(ids.cpu(), w_ids)
    dy = torch.randn(tokens, width, generator=gen, device="cuda")
    got = _backward(t, fan, dy, kept)
    want = torch.autograd.grad(want, list(leaves.values()), dy.double())
    for name, w in zip(leaves, want):
        assert float((got[name].double() - w).abs().max()) < 0.02 * float(w.abs().max()), name


def test_a_captured_layer_follows_new_inputs():
    """Decoding and a training step in graphs: replays, with eager work between them, match eager runs."""
    fan = 2
    for tokens in (1, 48, 300):
        gen = _gen(tokens)
        t = _layer(gen, tokens, 256, 512, 8)
        dy = torch.randn(tokens, 256, generator=gen, device="cuda")

        def step():
            y, kept = _forward(t, fan)
            return [y, kept[1], kept[2], kept[8]] + list(_backward(t, fan, dy, kept).values())

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for i in range(4):
            t["x"].copy_(ref.normal(gen, tokens, 256))
            dy.copy_(torch.randn(tokens, 256, generator=gen, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            for have, want in zip([o.clone() for o in out], step()):
                assert torch.equal(have, want), (tokens, i)


def test_two_graphs_of_one_pool_with_workspaces():
    """Parts of K and of the rows: two graphs whose workspaces may be the same memory, replayed in turn."""
    gen = _gen(77)
    cases = []
    for m, n, k in ((48, 1024, 4096), (130, 264, 2056)):
        assert g.lib().gemm_f16_fused_workspace(m, n, k) > 0
        a, b, res = ref.normal(gen, m, k), ref.normal(gen, n, k, std=k**-0.5), ref.normal(gen, m, n)
        dy, pre = ref.normal(gen, 40 * m, n), ref.normal(gen, 40 * m, n)
        assert g.lib().gemm_f16_fused_grad_workspace(40 * m, n) > 0
        cases.append((a, lambda a=a, b=b, res=res, dy=dy, pre=pre: [g.gemm_f16_fused_nt(a, b, act="silu", residual=res),
                                                                   *g.gemm_f16_fused_grad(dy, pre, act="silu")]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _, call in cases:
            call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, pool = [], torch.cuda.graph_pool_handle()
    for _, call in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = call()
        graphs.append((graph, out))
    for i in range(6):
        (a, call), (graph, out) = cases[i % 2], graphs[i % 2]
        a.copy_(ref.normal(gen, *a.shape))
        graph.replay()
        torch.cuda.synchronize()
        for have, want in zip([o.clone() for o in out], call()):
            assert torch.equal(have, want), i


def test_calls_on_streams_of_their_own():
    gen = _gen(31)
    calls = []
    for m in (3, 40, 70, 200):
        a, b = ref.normal(gen, m, 512), ref.normal(gen, 384, 512, std=0.05)
        bias, res = torch.randn(384, generator=gen, device="cuda"), ref.normal(gen, m, 384)
        calls.append(lambda a=a, b=b, bias=bias, res=res, **k: g.gemm_f16_fused_nt(a, b, bias, act="silu", residual=res, return_pre=True, **k))
    dy, pre = ref.normal(gen, 5000, 264), ref.normal(gen, 5000, 264)
    assert g.lib().gemm_f16_fused_grad_workspace(5000, 264) > 0
    calls.append(lambda **k: g.gemm_f16_fused_grad(dy, pre, act="gelu", **k))
    logits = torch.randn(500, 64, generator=gen, device="cuda")
    tilt = logits[0] * 0.1  # (here: the streams below do not wait for this one)
    calls.append(lambda **k: g.route(logits, 4, score="sigmoid", bias=tilt, groups=4, top_groups=2, **k))
    want = [[t.clone() for t in c()] for c in calls]
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for s in (side, third, side):
            got.append([c(stream=s) for c in calls])
            junk = [torch.full((1 << 18,), NAN, device="cuda") for _ in range(4)]
            del junk
        torch.cuda.synchronize()
        for runs in got:
            for have, expect in zip(runs, want):
                assert all(torch.equal(h, e) for h, e in zip(have, expect))


def test_refusals_of_tensors_on_the_gpu():
    h = torch.zeros(8, 16, dtype=F16, device="cuda")
    with pytest.raises(ValueError):
        g.gemm_f16_fused_nt(h.t(), h)
    with pytest.raises(ValueError):
        g.gemm_f16_fused_nt(h, h, residual=h)
    with pytest.raises(TypeError):
        g.gemm_f16_fused_nt(h, h, residual=torch.zeros(8, 8, device="cuda"))
    with pytest.raises(TypeError):
        g.gemm_f16_fused_nt(h, h, torch.zeros(8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        g.gemm_f16_fused_grad(h, act="silu")
    with pytest.raises(ValueError):
        g.gemm_f16_fused_grad(h, h[:4], act="silu")
    with pytest.raises(ValueError):
        g.route(h, 2, bias=torch.zeros(8, device="cuda"))
    x = torch.zeros(8, 8, dtype=F16, device="cuda")
    with pytest.raises(g.GemmError) as e:
        g.gemm_f16_fused_nt(x, x, out=x)
    assert e.value.status == g.EOVERLAP
