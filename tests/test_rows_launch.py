"""What the recurrence's launchers ask of the CUDA runtime, against a stand-in for it that is loaded in
front of the real one: two devices, failing queries, launches that are only counted. No GPU is touched."""
import json
import os
import subprocess
import sys

import pytest

from dense_linear_solvers_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Device-wide state as the runtime keeps it: a kernel's limit of dynamic shared memory belongs to the device
# that was current when it was raised, and a launch above the limit is refused.
STAND_IN = r"""
#include <map>
#include <utility>
#include <cuda_runtime_api.h>
static int device = 0, fail_queries = 0, queries = 0, launches = 0;
static std::map<std::pair<const void*, int>, int> limits;
static cudaError_t launched(const void* f, size_t shared) {
  auto at = limits.find({f, device});
  if (shared > static_cast<size_t>(at == limits.end() ? 48 << 10 : at->second))
    return cudaErrorInvalidValue;
  ++launches;
  return cudaSuccess;
}
extern "C" {
void stand_in_device(int d) { device = d; }
void stand_in_fail(int n) { fail_queries = n; }
int stand_in_queries() { return queries; }
int stand_in_launches() { return launches; }
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) limits[{f, device}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  ++queries;
  if (fail_queries > 0) { --fail_queries; return cudaErrorInitializationError; }
  *n = 304 / static_cast<int>(c->attrs[0].val.clusterDim.x);
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  return launched(f, c->dynamicSmemBytes);
}
cudaError_t __cudaGetKernel(void** kernel, const void* f) {
  *kernel = const_cast<void*>(f);
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(void* f, dim3, dim3, void**, size_t shared, cudaStream_t) {
  return launched(f, shared);
}
}
"""

CHILD = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
import dense_linear_solvers_gb300 as bs
from tests.test_rows_host import BACKWARD, FORWARD, P, call
lib = bs.lib()
out = {}
exec(sys.argv[3])
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    _build.build()
    at = tmp_path_factory.mktemp("stand_in")
    (at / "stand_in.cpp").write_text(STAND_IN)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.check_call(["g++", "-shared", "-fPIC", "-I", include, "-o", str(at / "stand_in.so"),
                           str(at / "stand_in.cpp")])
    return str(at / "stand_in.so")


def child(stand_in, code):
    out = subprocess.run([sys.executable, "-c", CHILD, stand_in, ROOT, code], capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    return json.loads(out.stdout.splitlines()[-1])


# every instance of a type: few and many sequences, equal and packed, aligned and not
CALLS = """
def calls():
    got = []
    for dtype, size in ((bs.BS_FP32, 4), (bs.BS_BF16, 2), (bs.BS_FP16, 2)):
        for off in (0, size):
            for batch, rows, offsets in ((2, 200, None), (400, 4000, None), (400, 4000, P[20])):
                for entry, args in ((lib.bs_grec_batched, FORWARD),
                                    (lib.bs_grec_backward_batched, BACKWARD)):
                    got.append(call(entry, args, dtype=dtype, x=P[0] + off, batch=batch, rows=rows,
                                    offsets=offsets))
    return got
"""


def test_a_second_device(stand_in):
    """The limit of shared memory is raised on each device."""
    got = child(stand_in, CALLS + """
for device in (0, 1, 0, 5, 200):
    fake.stand_in_device(device)
    out[device] = calls()
""")
    for device in ("0", "1", "5", "200"):
        assert set(got[device]) == {0}, (device, got[device])


def test_a_failed_query_is_not_kept(stand_in):
    """A call whose query fails says so; the next asks again, and an answer is asked for once a device."""
    got = child(stand_in, """
for name, entry, args in (("forward", lib.bs_grec_batched, FORWARD),
                          ("backward", lib.bs_grec_backward_batched, BACKWARD)):
    fake.stand_in_fail(1)
    first = call(entry, args)
    second = call(entry, args)
    asked = fake.stand_in_queries()
    third = call(entry, args)
    out[name] = [first, second, third, fake.stand_in_queries() - asked]
""")
    assert got == {"forward": [3, 0, 0, 0], "backward": [3, 0, 0, 0]}


def test_disjoint_windows_of_one_matrix_are_taken(stand_in):
    """Operands of one row distance may interleave as column windows; windows that share an element,
    in one row or around a row's end, or of another row distance may not."""
    got = child(stand_in, """
f, b = lib.bs_grec_batched, lib.bs_grec_backward_batched
one = dict(x=P[0], r=P[0] + 128, i=P[0] + 256, h=P[0] + 384, ldx=256, ldr=256, ldi=256, ldh=256)
first = dict(x=P[0] + 128, r=P[0] + 256, i=P[0] + 384, h=P[0], ldx=256, ldr=256, ldi=256, ldh=256)
grads = dict(dx=P[7], dr=P[7] + 128, di=P[7] + 256, lddx=192, lddr=192, lddi=192)
rest = dict(grads, lddx=256, lddr=256, lddi=256, dh=P[7] + 384, lddh=256)
before = fake.stand_in_launches()
out["taken"] = [call(f, FORWARD, **one), call(f, FORWARD, **first), call(b, BACKWARD, **grads),
                call(b, BACKWARD, **rest),
                # rows behind another operand's last one, whatever the distances
                call(f, FORWARD, h=P[0] + 200 * 128), call(f, FORWARD, h=P[0] + 200 * 128, ldh=96)]
out["launches"] = fake.stand_in_launches() - before
out["refused"] = [call(f, FORWARD, **dict(one, h=P[0] + 382)), call(f, FORWARD, **dict(one, h=P[0] + 386)),
                  call(f, FORWARD, **dict(first, h=P[0] + 2)), call(f, FORWARD, **dict(one, ldh=260)),
                  call(b, BACKWARD, **dict(rest, dh=P[7] + 256)),
                  call(f, FORWARD, h=P[0] + 200 * 128 - 2)]
out["launches after"] = fake.stand_in_launches() - before
""")
    assert got["taken"] == [0] * 6 and got["launches"] == 4 + 2 * 2
    assert got["refused"] == [1] * 6 and got["launches after"] == got["launches"]
