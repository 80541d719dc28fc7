"""A product's workspace follows from its sizes alone: no device is asked for, and the answer is the
same whatever number of compute units the current one has.  A stand-in for the two runtime calls that
could tell is put in front of the library; no GPU is needed."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STANDIN = """
static int calls, units, at;
void standin_set(int device, int n) { at = device; units = n; calls = 0; }
int standin_calls(void) { return calls; }
int hipGetDevice(int *device) { ++calls; *device = at; return 0; }
int hipDeviceGetAttribute(int *value, int attribute, int device) { ++calls; (void)attribute; (void)device; *value = units; return 0; }
"""
SIZES = [(512, 4096, 8192), (512, 4096, 4096), (1024, 1024, 4096), (128, 4096, 4096), (700, 300, 4096), (2048, 2048, 8192),
         (300, 4096, 16384), (48, 4096, 4096), (16384, 64, 4096), (128, 4096, 4097)]
PROGRAM = """
import ctypes, json, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # ahead of the library's own dependencies
import dense_fp16_gemm_f16_amd as g
lib = g.lib()
out = []
for device, units in enumerate((256, 32, 38, 64, 128, 304)):
    shim.standin_set(device, units)
    sizes = [lib.gemm_f16_fused_workspace(*s) for s in json.loads(sys.argv[2])]
    asked = shim.standin_calls()
    tile = lib.gemm_f16_select_tile(512, 4096, 8192)  # (of the current device, as documented: the stand-in is in use)
    out.append([sizes, asked, shim.standin_calls() > asked, tile])
print(json.dumps(out))
"""


def test_workspace_is_the_same_on_every_device(tmp_path):
    src, shim = tmp_path / "standin.c", tmp_path / "standin.so"
    src.write_text(STANDIN)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(shim), str(src)], check=True)
    run = subprocess.run([sys.executable, "-c", PROGRAM, str(shim), json.dumps(SIZES)], check=True, cwd=ROOT, capture_output=True, text=True)
    runs = json.loads(run.stdout.splitlines()[-1])
    assert all(r[2] for r in runs) and len({r[3] for r in runs}) > 1
    for sizes, asked, _, _ in runs:
        assert sizes == runs[0][0] and asked == 0
    assert any(runs[0][0])
