"""The binding of the gated delta rule and of the 8-bit calls enters the library on its operands' device,
whichever is current. No GPU is touched: the child process loads stand-ins for the entries and for the
runtime's device calls in front of the real ones, and the operands are torch's tensors without memory."""
import json
import os
import subprocess
import sys

from dense_linear_solvers_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_INS = r"""
extern "C" {
static int current = 0, seen[8], calls = 0;
int cudaGetDevice(int* d) { *d = current; return 0; }
int cudaSetDevice(int d) { current = d; return 0; }
int cudaGetDeviceCount(int* n) { *n = 0; return 100; }  // none: torch starts no context
int stand_in_current() { return current; }
int stand_in_calls() { return calls; }
int stand_in_seen(int k) { return seen[k]; }
#define ENTRY(name) int name(...) { seen[calls++ % 8] = current; return 0; }
ENTRY(bs_gdelta_batched)
ENTRY(bs_gdelta_backward_batched)
ENTRY(bs_gdelta_step_batched)
ENTRY(bs_gnorm_q8_batched)
ENTRY(bs_gemm_q8)
}
"""

CHILD = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
import warnings
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
sys.path.insert(0, sys.argv[2])
import dense_linear_solvers_gb300 as bs
with FakeTensorMode():
    new = lambda *s, **k: torch.empty(*s, device="cuda:1", **k)
    q, k, dq, dk = (new(2, 40, 1, 8) for _ in range(4))
    v, o, do, dv = (new(2, 40, 2, 8) for _ in range(4))
    g, beta, dg, db = (new(2, 40, 2) for _ in range(4))
    work, tape = new(1 << 20, dtype=torch.uint8), new(bs.bs_gdelta_tape(2, 8, 8, 2, 80), dtype=torch.uint8)
    state = new(2, 2, 8, 8)
    f, q8, s8 = new(5, 256), new(5, 256, dtype=torch.float8_e4m3fn), new(5, 2)
    w8, sw, y = new(64, 256, dtype=torch.float8_e4m3fn), new(1, 2), new(5, 64)
    there = torch.empty(5, 256, device="cuda:0")
    there8 = torch.empty(5, 256, device="cuda:0", dtype=torch.float8_e4m3fn)
    scales = torch.empty(5, 2, device="cuda:0")
bs.bs_gdelta_batched(q, k, v, g, beta, o, work, tape=tape, stream=0)
bs.bs_gdelta_backward_batched(q, k, v, g, beta, tape, do, dq, dk, dv, dg, db, work, stream=0)
bs.bs_gdelta_step_batched(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], state, o[:, 0], stream=0)
bs.bs_gnorm_q8_batched(f, q8, s8, stream=0)
bs.bs_gemm_q8(q8, s8, w8, sw, y, stream=0)
after, refused = fake.stand_in_current(), []
for call in (lambda: bs.bs_gemm_q8(there8, s8, w8, sw, y, stream=0),
             lambda: bs.bs_gnorm_q8_batched(f, q8, scales, stream=0)):
    try:
        call()
    except ValueError as e:
        refused.append(str(e))
bs.bs_gnorm_q8_batched(there, there8, scales, stream=0)
print(json.dumps({"seen": [fake.stand_in_seen(k) for k in range(fake.stand_in_calls())],
                  "after": after, "refused": refused}))
"""


def test_calls_run_on_their_operands_device(tmp_path):
    _build.build()
    source, library = tmp_path / "stand_ins.cpp", tmp_path / "stand_ins.so"
    source.write_text(STAND_INS)
    subprocess.check_call(["g++", "-shared", "-fPIC", "-o", str(library), str(source)])
    out = subprocess.run([sys.executable, "-W", "ignore", "-c", CHILD, str(library), ROOT],
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    got = json.loads(out.stdout.splitlines()[-1])
    assert got["seen"] == [1] * 5 + [0], got
    assert got["after"] == 0, got
    assert len(got["refused"]) == 2 and all("device" in r for r in got["refused"]), got
