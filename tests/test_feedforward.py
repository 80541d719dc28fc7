"""The feed-forward layer's host side: argument checks of the C entry points
(every call returns before the first HIP call), the binding's refusals, and
the definitions that the GPU tests compare against.  No GPU is needed."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from dense_fp16_gemm_f16_amd.feedforward import Epilogue, Routing
from tests import _codeobj
from tests import _feedforward as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G, H, W = (0x10000000 * i for i in range(1, 10))  # never dereferenced
BIG = 1 << 40
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _fused(m=8, n=16, k=32, a=A, b=B, c=C, act=0, bias_f32=0, out_f32=0, bias=None, residual=None, pre=None, ws=W, size=BIG,
           plain=False):
    e = Epilogue(act, bias_f32, out_f32, bias, residual, pre)
    return g.lib().gemm_f16_fused_nt(m, n, k, a, b, c, None if plain else ctypes.byref(e), ws, size, None)


@pytest.mark.parametrize("change, expect", [
    ({"m": -1}, g.EINVAL), ({"n": -1}, g.EINVAL), ({"k": -1}, g.EINVAL), ({"m": 1 << 30}, g.EINVAL), ({"n": 1 << 30}, g.EINVAL),
    ({"k": 1 << 22}, g.EINVAL), ({"m": 1 << 24, "n": 1 << 23}, g.EINVAL),
    ({"act": -1}, g.EINVAL), ({"act": 5}, g.EINVAL), ({"bias_f32": 2}, g.EINVAL), ({"out_f32": -1}, g.EINVAL),
    ({"size": -1}, g.EINVAL),
    ({"a": None}, g.ENULL), ({"b": None}, g.ENULL), ({"c": None}, g.ENULL),
    ({"a": A + 1}, g.EALIGN), ({"c": C + 1}, g.EALIGN), ({"c": C + 2, "out_f32": 1}, g.EALIGN), ({"bias": D + 1}, g.EALIGN),
    ({"bias": D + 2, "bias_f32": 1}, g.EALIGN), ({"residual": D + 2, "out_f32": 1}, g.EALIGN), ({"pre": D + 1}, g.EALIGN),
    ({"c": A + 16}, g.EOVERLAP), ({"c": B}, g.EOVERLAP), ({"pre": A}, g.EOVERLAP), ({"pre": C}, g.EOVERLAP),
    ({"bias": C + 2}, g.EOVERLAP), ({"residual": C + 2}, g.EOVERLAP), ({"residual": C, "pre": C + 32}, g.EOVERLAP),
    ({"pre": D, "residual": D}, g.EOVERLAP),
    ({"m": 0, "a": None, "c": None}, g.OK), ({"n": 0, "b": None, "c": None}, g.OK), ({"m": 0, "plain": True}, g.OK),
])
def test_fused_checks(change, expect):
    assert _fused(**change) == expect


@pytest.mark.parametrize("change, expect", [
    ({"m": -1}, g.EINVAL), ({"n": 1 << 30}, g.EINVAL), ({"act": 5}, g.EINVAL), ({"dy_f32": 2}, g.EINVAL), ({"size": 0}, g.EINVAL),
    ({"dy": None}, g.ENULL), ({"pre": None}, g.ENULL), ({"ws": None}, g.ENULL), ({"ws": W + 4}, g.EALIGN),
    ({"dy": A + 2, "dy_f32": 1}, g.EALIGN), ({"dbias": D + 2}, g.EALIGN), ({"dz": A + 2}, g.EOVERLAP), ({"dz": B}, g.EOVERLAP),
    ({"dz": A, "dy_f32": 1}, g.EOVERLAP), ({"dbias": A}, g.EOVERLAP), ({"dbias": C}, g.EOVERLAP), ({"ws": B}, g.EOVERLAP),
    ({"n": 0}, g.OK), ({"dz": None, "dbias": None}, g.OK), ({"m": 0, "dbias": None}, g.OK),
])
def test_fused_grad_checks(change, expect):
    v = {"m": 4096, "n": 64, "dy": A, "dy_f32": 0, "pre": B, "act": 4, "dz": C, "dbias": D, "ws": W, "size": BIG, **change}
    assert g.lib().gemm_f16_fused_grad(*v.values(), None) == expect


def test_workspace_sizes():
    L = g.lib()
    for m, n, k in ((0, 0, 0), (1, 4096, 4096), (1000, 700, 64), ((1 << 30) - 1, 1, 8), (1, (1 << 30) - 1, 8)):
        assert 0 <= L.gemm_f16_fused_workspace(m, n, k) <= 1 << 30
        assert 0 <= L.gemm_f16_fused_grad_workspace(m, n) <= 1 << 33
    for bad in ((-1, 1, 1), (1, 1 << 30, 1), (1, 1, 1 << 22), (1 << 24, 1 << 23, 1)):
        assert L.gemm_f16_fused_workspace(*bad) == g.EINVAL
    assert L.gemm_f16_fused_grad_workspace(-1, 1) == g.EINVAL


def _route(tokens=4, experts=16, fan=2, logits=A, f32=1, bias=None, score=0, groups=1, top_groups=1, group_top=1,
           renormalize=1, scale=1.0, ids=C, gates=D, null=False):
    r = Routing(score, groups, top_groups, group_top, renormalize, scale)
    return g.lib().gemm_f16_route(tokens, experts, fan, logits, f32, bias, None if null else ctypes.byref(r), ids, gates, None)


@pytest.mark.parametrize("change, expect", [
    ({"tokens": -1}, g.EINVAL), ({"tokens": 1 << 30}, g.EINVAL), ({"experts": 0}, g.EINVAL), ({"experts": 2049}, g.EINVAL),
    ({"fan": 0}, g.EINVAL), ({"fan": 33, "experts": 64}, g.EINVAL), ({"fan": 17}, g.EINVAL), ({"f32": 2}, g.EINVAL),
    ({"score": 2}, g.EINVAL), ({"groups": 0}, g.EINVAL), ({"groups": 3}, g.EINVAL), ({"groups": 128, "experts": 128}, g.EINVAL),
    ({"groups": 4, "top_groups": 0}, g.EINVAL), ({"groups": 4, "top_groups": 5}, g.EINVAL), ({"group_top": 0}, g.EINVAL),
    ({"group_top": 3}, g.EINVAL), ({"groups": 8, "top_groups": 1, "fan": 3}, g.EINVAL), ({"renormalize": 2}, g.EINVAL),
    ({"scale": float("inf")}, g.EINVAL), ({"scale": float("nan")}, g.EINVAL),
    ({"null": True}, g.ENULL), ({"logits": None}, g.ENULL), ({"ids": None}, g.ENULL), ({"gates": None}, g.ENULL),
    ({"logits": A + 2}, g.EALIGN), ({"bias": B + 2}, g.EALIGN), ({"ids": C + 2}, g.EALIGN),
    ({"ids": A}, g.EOVERLAP), ({"gates": C}, g.EOVERLAP), ({"bias": D}, g.EOVERLAP),
    ({"tokens": 0, "logits": None, "ids": None}, g.OK),
])
def test_route_checks(change, expect):
    assert _route(**change) == expect


@pytest.mark.parametrize("change, expect", [
    ({"tokens": -1}, g.EINVAL), ({"fan": 17}, g.EINVAL), ({"f32": -1}, g.EINVAL), ({"dlogits": None}, g.ENULL),
    ({"ids": None}, g.ENULL), ({"dgates": None}, g.ENULL), ({"r": None}, g.ENULL), ({"dlogits": A}, g.EOVERLAP),
    ({"dlogits": E + 2}, g.EALIGN), ({"tokens": 0}, g.OK),
])
def test_route_grad_checks(change, expect):
    r = Routing(0, 1, 1, 1, 1, 1.0)
    v = {"tokens": 4, "experts": 16, "fan": 2, "logits": A, "f32": 1, "ids": C, "dgates": D, "r": ctypes.byref(r), "dlogits": E,
         **change}
    assert g.lib().gemm_f16_route_grad(*v.values(), None) == expect


COMBINE = {"tokens": 4, "fan": 2, "n": 16, "groups": 3, "rows": A, "rows_f32": 0, "inverse": B, "offsets": C, "gates": D,
           "residual": E, "y": F, "y_f32": 0}


@pytest.mark.parametrize("change, expect", [
    ({"tokens": -1}, g.EINVAL), ({"fan": 0}, g.EINVAL), ({"n": 1 << 30}, g.EINVAL), ({"tokens": 1 << 29, "fan": 2}, g.EINVAL),
    ({"groups": 0}, g.EINVAL), ({"rows_f32": 2}, g.EINVAL), ({"y_f32": -1}, g.EINVAL),
    ({"rows": None}, g.ENULL), ({"inverse": None}, g.ENULL), ({"offsets": None}, g.ENULL), ({"y": None}, g.ENULL),
    ({"rows": A + 2, "rows_f32": 1}, g.EALIGN), ({"gates": D + 2}, g.EALIGN), ({"offsets": C + 2}, g.EALIGN),
    ({"y": A}, g.EOVERLAP), ({"y": B}, g.EOVERLAP), ({"y": D}, g.EOVERLAP), ({"residual": F + 2}, g.EOVERLAP),
    ({"tokens": 0}, g.OK), ({"n": 0}, g.OK),
])
def test_combine_checks(change, expect):
    assert g.lib().gemm_f16_combine_rows(*{**COMBINE, **change}.values(), None) == expect


COMBINE_GRAD = {"tokens": 4, "fan": 2, "n": 16, "groups": 3, "dy": E, "dy_f32": 0, "rows": A, "rows_f32": 0, "inverse": B,
                "offsets": C, "gates": D, "drows": F, "drows_f32": 0, "dgates": G}


@pytest.mark.parametrize("change, expect", [
    ({"tokens": -1}, g.EINVAL), ({"fan": 0}, g.EINVAL), ({"dy_f32": 2}, g.EINVAL), ({"drows_f32": 2}, g.EINVAL),
    ({"dy": None}, g.ENULL), ({"rows": None}, g.ENULL), ({"inverse": None}, g.ENULL), ({"dgates": G + 2}, g.EALIGN),
    ({"drows": A}, g.EOVERLAP), ({"drows": E}, g.EOVERLAP), ({"dgates": D}, g.EOVERLAP), ({"drows": G}, g.EOVERLAP),
    ({"tokens": 0}, g.OK), ({"drows": None, "dgates": None}, g.OK), ({"n": 0, "dgates": None}, g.OK),
])
def test_combine_grad_checks(change, expect):
    assert g.lib().gemm_f16_combine_rows_grad(*{**COMBINE_GRAD, **change}.values(), None) == expect


def test_other_architectures_are_refused():
    code = ("import ctypes\nimport dense_fp16_gemm_f16_amd as g\nfrom tests import test_feedforward as t\n"
            "r = t.Routing(0, 1, 1, 1, 1, 1.0)\n"
            "assert t._fused() == t._route() == g.EDEVICE\n"
            "assert g.lib().gemm_f16_fused_grad(8, 8, t.A, 0, t.B, 4, t.C, None, None, 0, None) == g.EDEVICE\n"
            "assert g.lib().gemm_f16_route_grad(4, 16, 2, t.A, 1, t.C, t.D, ctypes.byref(r), t.E, None) == g.EDEVICE\n"
            "assert g.lib().gemm_f16_combine_rows(*t.COMBINE.values(), None) == g.EDEVICE\n"
            "assert g.lib().gemm_f16_combine_rows_grad(*t.COMBINE_GRAD.values(), None) == g.EDEVICE\n")
    env = {**os.environ, "GEMM_F16_TEST_ARCH": "gfx942"}
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, env=env)


def _registers(token):
    """Accumulator registers of an operand: a7, or a[4:7]."""
    m = re.match(r"a\[(\d+):(\d+)\]$", token) or re.match(r"a(\d+)()$", token)
    return set(range(int(m[1]), int(m[2] or m[1]) + 1)) if m else set()


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump not installed")
def test_accumulators_rest_behind_their_mfmas(tmp_path):
    """The large tiles' MFMAs are inline asm, so the compiler leaves no wait before it reads or
    moves what they write: no such move may stand within 18 wait states behind one (16x16x32: 8
    passes of 4 cycles and a few more) in those kernels of the products with an epilogue."""
    with open(g.LIB_PATH, "rb") as f:
        blob = f.read()
    kernels, bad = set(), []
    for i, (triple, obj) in enumerate(_codeobj._bundles(blob)):
        if "gfx950" not in triple or b"fused_" not in obj:
            continue
        path = tmp_path / f"co{i}.o"
        path.write_bytes(obj)
        asm = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True, check=True).stdout
        name, age, recent = None, 0, []
        for line in asm.splitlines():
            head = re.match(r"[0-9a-f]+ <(\S+)>:", line)
            if head:
                name, recent = head[1], []
                kernels.add(name)
                continue
            op, _, rest = line.split("//")[0].strip().partition(" ")
            if not re.search("fused_(tile|direct|walk)_kernel", name or "") or not op:
                continue
            args = [x.strip() for x in rest.split(",")]
            age += 1 + (int(args[0], 0) if op == "s_nop" else 0)
            if op.startswith("v_mfma"):
                recent = [r for r in recent if age - r[0] < 40] + [(age, _registers(args[0]))]
            elif "accvgpr" in op:
                touched = set().union(*map(_registers, args))
                bad += [(name, line.strip()) for at, r in recent if r & touched and age - at < 18]
    assert any("fused_walk_kernel" in k for k in kernels) and any("fused_tile_kernel" in k for k in kernels)
    assert not bad, (len(bad), bad[:4])


def _h(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: g.gemm_f16_fused_nt(_h(4, 8), _h(8, 8)),                        # not on a GPU
    lambda: g.gemm_f16_fused_grad(_h(4, 8)),
    lambda: g.route(_h(4, 8), 2),
    lambda: g.route_grad(_h(4, 8), _i(4, 2), torch.zeros(4, 2)),
    lambda: g.combine_rows(_h(4, 8), _i(4), _i(3), 2),
    lambda: g.combine_rows_grad(_h(2, 8), _h(4, 8), _i(4), _i(3), torch.zeros(2, 2)),
    lambda: g.gemm_f16_fused_nt(_h(4, 8), _h(8, 8), act="tanh"),            # no such activation
    lambda: g.gemm_f16_fused_grad(_h(4, 8), act="elu"),
    lambda: g.route(_h(4, 8), 2, score="relu"),
    lambda: g.gemm_f16_fused_nt(_h(8), _h(8, 8)),                           # shapes
    lambda: g.route(_h(8), 2),
    lambda: g.combine_rows(_h(5, 8), _i(5), _i(3), 2),
    lambda: g.combine_rows(_h(4, 8), _i(4), _i(1), 2),
    lambda: g.combine_rows(_h(4, 8), _i(4), _i(3), 0),
])
def test_binding_refuses_shapes_and_devices(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: g.gemm_f16_fused_nt(torch.zeros(4, 8), _h(8, 8)),
    lambda: g.gemm_f16_fused_nt(_h(4, 8), _h(8, 8), out_dtype=torch.bfloat16),
    lambda: g.gemm_f16_fused_grad(torch.zeros(4, 8, dtype=torch.bfloat16)),
    lambda: g.route(torch.zeros(4, 8, dtype=torch.float64), 2),
    lambda: g.combine_rows(torch.zeros(4, 8, dtype=torch.int32), _i(4), _i(3), 2),
    lambda: g.combine_rows(_h(4, 8), _i(4), _i(3), 2, out_dtype=torch.float64),
])
def test_binding_refuses_types(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("name", ref.ACTS)
def test_activation_gradients_against_differences(name):
    z = torch.linspace(-6, 6, 97, dtype=torch.float64) + 0.013
    slope = (ref.act(name, z + 1e-6) - ref.act(name, z - 1e-6)) / 2e-6
    assert torch.allclose(ref.act_grad(name, z), slope, atol=1e-8)
    if name in ("gelu", "gelu_tanh", "silu"):
        assert float(slope.abs().max()) < ref.SLOPE
        torch_form = {"gelu": lambda x: torch.nn.functional.gelu(x), "silu": torch.nn.functional.silu,
                      "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[name]
        assert torch.allclose(ref.act(name, z), torch_form(z), atol=1e-12)


def test_routing_definition_on_worked_cases():
    inf, nan = float("inf"), float("nan")
    l = torch.tensor([[1.0, 3.0, 3.0, 2.0], [-inf, -inf, -inf, -inf], [nan, 0.0, -inf, -1.0], [inf, 0.0, inf, 1.0]])
    ids, gates = ref.route(l, 2)
    assert ids.tolist() == [[1, 2], [-1, -1], [1, 3], [0, 2]]
    assert gates[0].tolist() == [0.5, 0.5] and gates[1].tolist() == [0, 0] and gates[3].tolist() == [0.5, 0.5]
    assert torch.allclose(gates[2], torch.softmax(torch.tensor([0.0, -1.0], dtype=torch.float64), 0))
    ids, gates = ref.route(l[:1], 2, bias=torch.tensor([2.0, 0.0, -inf, 0.0]), renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 1]]
    assert torch.allclose(gates, 2 * torch.softmax(l[:1].double(), 1)[:, :2])
    # two groups of two: sums of two sigmoids 1.5 and 1.3, largest .8 and .9
    l = torch.logit(torch.tensor([[0.8, 0.7, 0.9, 0.4]], dtype=torch.float64))
    assert ref.route(l, 1, score="sigmoid", groups=2, group_top=2)[0].tolist() == [[0]]
    assert ref.route(l, 1, score="sigmoid", groups=2, group_top=1)[0].tolist() == [[2]]


def test_combination_definition_on_a_worked_case():
    rows = torch.arange(8.0).view(4, 2)
    inverse = torch.tensor([2, 0, 1, 3])
    gates = torch.tensor([[0.5, 2.0], [1.0, 7.0]])
    y, _ = ref.combine(rows, inverse, 3, 2, gates, torch.ones(2, 2))
    assert y.tolist() == [[1 + 2.0 + 0.0, 1 + 2.5 + 2.0], [1 + 2.0, 1 + 3.0]]
    d = torch.tensor([[1.0, -1.0], [2.0, 0.5]])
    leaf_r, leaf_g = rows.double().requires_grad_(), gates.double().requires_grad_()
    y, _ = ref.combine(leaf_r, inverse, 3, 2, leaf_g, None)
    want = torch.autograd.grad(y, (leaf_r, leaf_g), d.double())
    got = ref.combine_grad(d, rows, inverse, 3, gates)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
