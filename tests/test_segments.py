"""The segmented products' host side: argument checks of the C entry points
(every call returns before the first HIP call), workspace sizes, the
binding's refusals, and the definitions that the GPU tests compare against.
No GPU is needed."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import dense_fp16_gemm_f16_amd as g
from tests import _segments as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, O, I, W = (0x10000000 * i for i in range(1, 7))  # never dereferenced
BIG = 1 << 40


def _nt(rows=8, groups=2, n=16, k=16, a=A, a_rows=8, b=B, offsets=O, index=I, fan=1, c=C, f32=0):
    return g.lib().gemm_f16_grouped_nt(rows, groups, n, k, a, a_rows, b, offsets, index, fan, c, f32, None)


@pytest.mark.parametrize("change, expect", [
    ({"rows": -1}, g.EINVAL), ({"rows": 1 << 30}, g.EINVAL), ({"n": -1}, g.EINVAL), ({"n": 1 << 30}, g.EINVAL),
    ({"k": -1}, g.EINVAL), ({"k": 1 << 22}, g.EINVAL), ({"groups": 0}, g.EINVAL), ({"groups": (1 << 20) + 1}, g.EINVAL),
    ({"rows": 1 << 24, "n": 1 << 23, "a_rows": 1 << 24}, g.EINVAL), ({"groups": 1 << 20, "n": 1 << 20, "k": 1 << 10}, g.EINVAL),
    ({"fan": 0}, g.EINVAL), ({"f32": 2}, g.EINVAL), ({"f32": -1}, g.EINVAL), ({"a_rows": -1}, g.EINVAL),
    ({"index": None, "a_rows": 7}, g.EINVAL),
    ({"a": None}, g.ENULL), ({"b": None}, g.ENULL), ({"c": None}, g.ENULL), ({"offsets": None}, g.ENULL),
    ({"a": A + 1}, g.EALIGN), ({"b": B + 1}, g.EALIGN), ({"c": C + 1}, g.EALIGN), ({"c": C + 2, "f32": 1}, g.EALIGN),
    ({"offsets": O + 2}, g.EALIGN), ({"index": I + 2}, g.EALIGN),
    ({"c": A + 16}, g.EOVERLAP), ({"c": B}, g.EOVERLAP), ({"c": O}, g.EOVERLAP), ({"c": I}, g.EOVERLAP),
    ({"rows": 0, "a_rows": 0, "a": None, "b": None, "c": None, "offsets": None, "index": None}, g.OK),
    ({"n": 0, "c": None}, g.OK),
])
def test_grouped_nt_checks(change, expect):
    assert _nt(**change) == expect


@pytest.mark.parametrize("kind", ["nn", "tn"])
@pytest.mark.parametrize("change, expect", [
    ({"n": 1 << 25}, g.EINVAL), ({"rows": -1}, g.EINVAL), ({"groups": 0}, g.EINVAL), ({"k": 1 << 22}, g.EINVAL),
    ({"a": None}, g.ENULL), ({"offsets": None}, g.ENULL), ({"c": C + 2, "f32": 1}, g.EALIGN), ({"c": B}, g.EOVERLAP),
    ({"n": 0}, g.OK),
])
def test_grouped_gradient_checks(kind, change, expect):
    v = {"rows": 8, "groups": 2, "n": 16, "k": 16, "a": A, "b": B, "offsets": O, "c": C, "f32": 0, **change}
    call = getattr(g.lib(), "gemm_f16_grouped_" + kind)
    assert call(v["rows"], v["groups"], v["n"], v["k"], v["a"], v["b"], v["offsets"], v["c"], v["f32"], None) == expect


def _tn_ws(rows=9000, groups=2, n=64, k=128, a=A, b=B, offsets=O, c=C, f32=0, ws=W, size=BIG):
    return g.lib().gemm_f16_grouped_tn_ws(rows, groups, n, k, a, b, offsets, c, f32, ws, size, None)


@pytest.mark.parametrize("change, expect", [
    ({"rows": -1}, g.EINVAL), ({"groups": 0}, g.EINVAL), ({"n": 1 << 25}, g.EINVAL), ({"f32": 2}, g.EINVAL),
    ({"size": 4}, g.EINVAL), ({"ws": None}, g.ENULL), ({"a": None}, g.ENULL), ({"ws": W + 4}, g.EALIGN),
    ({"c": W}, g.EOVERLAP), ({"ws": A}, g.EOVERLAP), ({"ws": O}, g.EOVERLAP), ({"n": 0, "size": 0, "ws": None}, g.OK),
])
def test_grouped_tn_ws_checks(change, expect):
    assert _tn_ws(**change) == expect


def test_grouped_tn_workspace_sizes():
    size = g.lib().gemm_f16_grouped_tn_workspace
    assert size(16384, 1, 512, 512) >= 2 * 512 * 512 * 4           # few tiles, many rows: split
    for whole in ((100, 1, 512, 512), (16384, 8, 2048, 4096), (0, 4, 64, 64), (16384, 4, 0, 64), (16384, 4, 64, 0)):
        assert size(*whole) == 0
    for rows in (256, 5000, (1 << 30) - 1):
        for groups, n, k in ((1, 1, 1), (3, 61, 75), (7, 700, 500), (1 << 20, 8, 8), (1, 100000, 64)):
            assert 0 <= size(rows, groups, n, k) <= 512 * 65536
    for bad in ((-1, 1, 8, 8), (1 << 30, 1, 8, 8), (8, 0, 8, 8), (8, 1, 1 << 25, 8), (8, 1, 8, 1 << 22)):
        assert size(*bad) == g.EINVAL


@pytest.mark.parametrize("change, expect", [
    ({"rows": -1}, g.EINVAL), ({"rows": 1 << 30}, g.EINVAL), ({"groups": 0}, g.EINVAL), ({"groups": 2049}, g.EINVAL),
    ({"id_bytes": 2}, g.EINVAL), ({"size": 3}, g.EINVAL),
    ({"ids": None}, g.ENULL), ({"order": None}, g.ENULL), ({"offsets": None}, g.ENULL), ({"ws": None}, g.ENULL),
    ({"ids": A + 2}, g.EALIGN), ({"ids": A + 4, "id_bytes": 8}, g.EALIGN), ({"ws": W + 4}, g.EALIGN),
    ({"order": B}, g.EOVERLAP), ({"inverse": A}, g.EOVERLAP), ({"offsets": W}, g.EOVERLAP),
])
def test_group_rows_checks(change, expect):
    v = {"rows": 100000, "groups": 64, "ids": A, "id_bytes": 4, "order": C, "inverse": B, "offsets": O, "ws": W, "size": BIG, **change}
    rc = g.lib().gemm_f16_group_rows(v["rows"], v["groups"], v["ids"], v["id_bytes"], v["order"], v["inverse"],
                                     v["offsets"], v["ws"], v["size"], None)
    assert rc == expect


LORA = {"rows": 8, "n": 16, "k": 32, "adapters": 3, "rank": 4, "x": A, "w": B, "down": C, "up": O, "ids": I,
        "order": I + 0x1000, "offsets": I + 0x2000, "scale": I + 0x3000, "y": W, "ws": 0x70000000, "size": BIG}


@pytest.mark.parametrize("change, expect", [
    ({"rows": -1}, g.EINVAL), ({"n": 1 << 30}, g.EINVAL), ({"k": 1 << 22}, g.EINVAL), ({"adapters": 0}, g.EINVAL),
    ({"rank": 0}, g.EINVAL), ({"rank": 4097}, g.EINVAL), ({"size": 4}, g.EINVAL),
    ({"x": None}, g.ENULL), ({"up": None}, g.ENULL), ({"ids": None}, g.ENULL), ({"ws": None}, g.ENULL),
    ({"y": W + 1}, g.EALIGN), ({"scale": I + 0x3002}, g.EALIGN), ({"ws": 0x70000004}, g.EALIGN),
    ({"y": A}, g.EOVERLAP), ({"y": C}, g.EOVERLAP), ({"ws": W}, g.EOVERLAP), ({"ws": B}, g.EOVERLAP),
    ({"rows": 0}, g.OK), ({"n": 0}, g.OK),
])
def test_lora_checks(change, expect):
    v = {**LORA, **change}
    assert g.lib().gemm_f16_lora_nt(*(v[x] for x in LORA), None) == expect


def test_workspace_sizes():
    L = g.lib()
    assert L.gemm_f16_group_rows_workspace(100, 8) == 0  # one workgroup sorts them
    assert L.gemm_f16_group_rows_workspace(1 << 20, 64) >= 65 * 4
    for rows in (0, 1, 100, 1 << 20, (1 << 30) - 1):
        assert 0 <= L.gemm_f16_group_rows_workspace(rows, 2048) <= 256 * 2049 * 4
    for bad in ((-1, 4), (1 << 30, 4), (10, 0), (10, 2049)):
        assert L.gemm_f16_group_rows_workspace(*bad) == g.EINVAL
    assert L.gemm_f16_lora_workspace(8, 8, 8, 0, 4) == g.EINVAL
    assert L.gemm_f16_lora_workspace(8, 8, 8, 2, 4) >= 8 * 4 * 4


def test_other_architectures_are_refused():
    code = ("import dense_fp16_gemm_f16_amd as g\n"
            "from tests import test_segments as t\n"
            "assert t._nt() == g.EDEVICE\n"
            "assert g.lib().gemm_f16_lora_nt(*t.LORA.values(), None) == g.EDEVICE\n"
            "assert g.lib().gemm_f16_group_rows(8, 2, t.A, 4, t.C, t.B, t.O, None, 0, None) == g.EDEVICE\n")
    env = {**os.environ, "GEMM_F16_TEST_ARCH": "gfx942"}
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, env=env)


def _h(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("call", [
    lambda: g.group_rows(_i(8), 4),                                                    # not on a GPU
    lambda: g.gemm_f16_grouped_nt(_h(4, 8), _h(2, 8, 8), _i(3)),
    lambda: g.gemm_f16_grouped_nn(_h(4, 8), _h(2, 8, 8), _i(3)),
    lambda: g.gemm_f16_grouped_tn(_h(4, 8), _h(4, 8), _i(3)),
    lambda: g.gemm_f16_lora_nt(_h(4, 8), _h(8, 8), _h(2, 4, 8), _h(2, 8, 4), _i(4), _i(4), _i(3)),
    lambda: g.gemm_f16_grouped_nt(_h(4, 8), _h(8, 8), _i(3)),                          # b of two dimensions
    lambda: g.gemm_f16_grouped_tn(_h(4, 8), _h(2, 4, 8), _i(3)),                       # b of three
])
def test_binding_refuses_shapes_and_devices(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: g.group_rows(torch.zeros(8), 4),
    lambda: g.gemm_f16_grouped_nt(torch.zeros(4, 8), _h(2, 8, 8), _i(3)),
    lambda: g.gemm_f16_grouped_nt(_h(4, 8), _h(2, 8, 8), _i(3), out_dtype=torch.bfloat16),
])
def test_binding_refuses_types(call):
    with pytest.raises(TypeError):
        call()


def test_definitions_agree_on_a_worked_case():
    """Two experts, three rows, by hand; the gradients against differences in 64 bits."""
    order, inverse, offsets = ref.group_rows([1, 7, 0, 1], 2)
    assert order.tolist() == [2, 0, 3, 1] and inverse.tolist() == [1, 3, 0, 2] and offsets.tolist() == [0, 1, 3]
    gen = torch.Generator().manual_seed(3)
    a, w, up = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 4), (2, 5, 4), (3, 5)))
    off = [0, 1, 3]
    c, _, _ = ref.grouped("nt", a, w, off)
    assert torch.allclose(c[0], w[0] @ a[0]) and torch.allclose(c[2], w[1] @ a[2])
    da, _, _ = ref.grouped("nn", up, w, off)
    dw, _, _ = ref.grouped("tn", up, a, off)
    for grad, t, at in ((da, a, (1, 2)), (da, a, (0, 3)), (dw, w, (0, 4, 1)), (dw, w, (1, 0, 3))):
        moved = []
        for step in (1e-4, -1e-4):
            u = t.clone()
            u[at] += step
            y, _, _ = ref.grouped("nt", u if t is a else a, u if t is w else w, off)
            moved.append((y * up).sum())
        assert abs((moved[0] - moved[1]) / 2e-4 - grad[at]) < 1e-8
    y, _ = ref.lora(a, w[0], w[:, :2], torch.ones(2, 5, 2), torch.tensor([1, -1, 0]), torch.tensor([2.0, 0.5]))
    assert torch.allclose(y[1], w[0] @ a[1])
    assert torch.allclose(y[0], w[0] @ a[0] + 0.5 * (w[1, :2] @ a[0]).sum())
    assert torch.allclose(y[2], w[0] @ a[2] + 2.0 * (w[0, :2] @ a[2]).sum())
