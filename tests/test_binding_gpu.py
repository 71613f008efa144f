"""The native binding against a stand-in for the library."""
import os
import shutil
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = ["sq_quant_act_e4m3_block", "sq_smooth_quant_weight_e4m3_block", "sq_w8a8_linear_e4m3_block",
         "sq_w8a8_linear_grouped", "sq_w8a8_linear_grouped_e4m3", "sq_w8a8_linear_grouped_e4m3_block"]

USE = """
import sys, torch
import w8a8_post_quantization_channel_b200 as sq
sq._marshal().init(sys.argv[1])
u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
f = lambda *s: torch.zeros(s, device="cuda")
off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
sq.sq_quant_act_e4m3_block(f(4, 256))
sq.sq_smooth_quant_weight_e4m3_block(f(256, 256))
sq.sq_w8a8_linear_e4m3_block(u(4, 256), f(4, 2), u(256, 256), f(2, 2))
sq.sq_w8a8_linear_grouped(u(4, 256).to(torch.int8), f(4), u(1, 256, 256).to(torch.int8), f(1, 256), off)
sq.sq_w8a8_linear_grouped_e4m3(u(4, 256), f(4), u(1, 256, 256), f(1, 256), off)
sq.sq_w8a8_linear_grouped_e4m3_block(u(4, 256), f(4, 2), u(1, 256, 256), f(1, 2, 2), off)
print("six calls")
"""


def test_calls_release_the_interpreter(tmp_path):
    # a launch can wait for room in the queue: other threads go on meanwhile,
    # as under the ctypes calls.  The stand-in's calls fail if they hold the lock
    assert shutil.which("gcc")
    src = tmp_path / "held.c"
    src.write_text("int PyGILState_Check(void);\n" +
                   "".join(f"int {name}(void) {{ return PyGILState_Check() ? 3 : 0; }}\n" for name in CALLS))
    so = tmp_path / "held.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    r = subprocess.run([sys.executable, "-c", USE, str(so)], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "six calls" in r.stdout, r.stderr[-2000:]
