"""The dense and the segmented entry points have one device gate: what the
environment says after the library has loaded changes neither."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_test_architecture_is_read_as_the_library_loads():
    code = ("import os\n"
            "import dense_fp16_gemm_f16_amd as g\n"
            "from tests import test_segments as t\n"
            "g.lib()\n"
            "os.environ['GEMM_F16_TEST_ARCH'] = 'gfx942'\n"
            "dense = g.gemm_f16_nt_raw(16, 16, 16, t.A, t.B, t.C)\n"
            "assert dense == g.EHIP, dense\n"
            "assert t._nt() == dense\n"
            "assert g.lib().gemm_f16_lora_nt(*t.LORA.values(), None) == dense\n"
            "assert g.lib().gemm_f16_group_rows(8, 2, t.A, 4, t.C, t.B, t.O, None, 0, None) == dense\n")
    # no device is visible, so that no call can reach one
    env = {**os.environ, "HIP_VISIBLE_DEVICES": "-1", "ROCR_VISIBLE_DEVICES": "-1"}
    env.pop("GEMM_F16_TEST_ARCH", None)
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, env=env)
