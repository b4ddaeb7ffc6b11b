"""The row operators' binding enters the library on its operands' device, whichever is current. No GPU is
touched: the child process loads stand-ins for the entries and for the runtime's device calls in front of
the real ones, and the operands are torch's tensors without memory."""
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
ENTRY(bs_grec_batched)
ENTRY(bs_grec_backward_batched)
ENTRY(bs_grec_step_batched)
ENTRY(bs_gnorm_batched)
ENTRY(bs_gnorm_backward_batched)
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
    x, r, i, h, lam = *(new(2, 40, 8) for _ in range(4)), new(8)
    tape, work = new(bs.bs_grec_tape_rows(2, 80), 8), new(1 << 16, dtype=torch.uint8)
    t, state = new(2, 8), new(2, 8)
    elsewhere = torch.empty(2, 40, 8, device="cuda:0")
bs.bs_grec_batched(x, r, i, lam, h, tape=tape, stream=0)
bs.bs_grec_backward_batched(x, r, i, lam, tape, h, x, r, i, lam, work, stream=0)
bs.bs_grec_step_batched(t, t, t, lam, state, t, stream=0)
bs.bs_gnorm_batched(x, h, stream=0)
bs.bs_gnorm_backward_batched(x, h, r, work, stream=0)
after = fake.stand_in_current()
try:
    bs.bs_gnorm_batched(x, elsewhere, stream=0)
    refused = ""
except ValueError as e:
    refused = str(e)
bs.bs_gnorm_batched(elsewhere, elsewhere, stream=0)
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
    assert "device" in got["refused"], got
