"""Each call as the very first of its process, in a CUDA graph's capture: what a kernel
asks of the device once is asked there."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import moe_expert_ffn_smoe_gb300 as smoe
torch.zeros(1, device="cuda")
u8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")  # ones
one = lambda *s: torch.ones(*s, device="cuda")
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
s = torch.cuda.Stream()
"""
END = """
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    call()
g.replay()
torch.cuda.synchronize()
assert smoe.smoe_last_device_status() == smoe.SMOE_OK
check()
print("fine")
"""
PRODUCT = """
need = smoe.smoe_experts_matmul_f8_workspace_bytes({R}, {R}, 2, {N}, 2048)
y, work, off = one({R}, {N}) * 5, u8(max(need, 16)), i32(0, {R} // 2, {R})
args = (u8({R}, 2048), one({R}, 16), {R}, None, 1, off, {R}, 2, u8(2, {N}, 2048), one(2, ({N} + 127) // 128, 16), {N}, 2048, y, 0, work, need)
call = lambda: smoe.smoe_experts_matmul_f8(*args, s)
check = lambda: torch.testing.assert_close(y, torch.full_like(y, 2048.0), rtol=0, atol=0)
"""
CALLS = {
    "routing": """
l, b, idx, w = one(5, 128), one(128), i32(*[7] * 40), one(40)
call = lambda: smoe.smoe_route_rows(l, 5, 128, 128, b, 1, 8, 4, 2, 8, 1, 2.0, idx, w, s)
check = lambda: (torch.testing.assert_close(idx.view(5, 8), i32(*range(8)).expand(5, 8)), torch.testing.assert_close(w, one(40) / 4))
""",
    "routing's gradient": """
l, idx, w, dw, d = one(5, 12), i32(*[3] * 5), one(5), one(5), one(5, 12) * 9
call = lambda: smoe.smoe_route_rows_backward(l, 5, 12, 12, 0, 1, 1, 1.0, idx, w, dw, d, s)
check = lambda: torch.testing.assert_close(d, one(5, 12) * 0)
""",
    "rows": """
x, q, sc = one(5, 512), u8(5, 256) * 0, one(5, 2) * 9
call = lambda: smoe.smoe_quantize_rows_f8(x, 0, 1, 5, 256, q, sc, s)
check = lambda: torch.testing.assert_close(q.view(torch.float8_e4m3fn).float(), torch.full((5, 256), 448.0, device="cuda"))
""",
    "matrices": """
x, q, sc, qt, st = one(2, 130, 144), u8(2, 130, 144) * 0, one(2, 2, 2), u8(2, 144, 130) * 0, one(2, 2, 2)
call = lambda: smoe.smoe_quantize_blocks_f8(x, 0, 2, 130, 144, q, sc, qt, st, s)
check = lambda: torch.testing.assert_close(qt.view(torch.float8_e4m3fn).float(), torch.full((2, 144, 130), 448.0, device="cuda"))
""",
    "few rows, split": PRODUCT.format(R=4, N=256),
    "few rows": PRODUCT.format(R=30, N=20000),
    "many rows": PRODUCT.format(R=3000, N=4096),
    "weights' gradient": """
dy, x, dw = one(40, 264).bfloat16(), one(40, 520).bfloat16(), one(2, 264, 520) * 5
off = i32(0, 10, 40)
call = lambda: smoe.smoe_experts_weight_grad(dy, x, off, 40, 2, 264, 520, 0, dw, 0, s)
check = lambda: torch.testing.assert_close(dw, torch.tensor([10.0, 30.0], device="cuda")[:, None, None].expand(2, 264, 520))
""",
}


@pytest.mark.parametrize("which", list(CALLS))
def test_the_first_call(which):
    r = subprocess.run([sys.executable, "-c", SETUP + CALLS[which] + END, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr[-2000:]
