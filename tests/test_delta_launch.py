"""What the launchers of the gated delta rule and of the 8-bit product ask of the CUDA runtime, against a stand-in
for it that is loaded in front of the real one: it notes every limit that is set and every kernel that would run, by
name. No GPU is touched."""
import json
import os
import subprocess
import sys

import pytest

from dense_linear_solvers_gb300 import _build
from tests.delta_forms import CHAINS, PACKED, PRODUCTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A launch above its kernel's limit of dynamic shared memory is refused, as by the runtime.
STAND_IN = r"""
#include <cstdint>
#include <cstdlib>
#include <cxxabi.h>
#include <map>
#include <string>
#include <cuda_runtime_api.h>
#include <dlfcn.h>
static std::map<const void*, std::string> names;
static std::map<const void*, int> limits;
static std::string notes;
static std::string name_of(const void* f) {
  int status = 0;
  char* plain = abi::__cxa_demangle(names[f].c_str(), nullptr, nullptr, &status);
  std::string s = status == 0 ? plain : names[f];
  std::free(plain);
  return s.substr(0, s.rfind(">(") + 1);
}
static cudaError_t launched(const void* f, dim3 grid, dim3 block, size_t shared, int cluster) {
  auto at = limits.find(f);
  if (shared > static_cast<size_t>(at == limits.end() ? 48 << 10 : at->second)) return cudaErrorInvalidValue;
  notes += "launch|" + name_of(f) + "|" + std::to_string(grid.x) + "|" + std::to_string(block.x) + "|" +
           std::to_string(shared) + "|" + std::to_string(cluster) + "\n";
  return cudaSuccess;
}
static int encode(...) { return 0; }
extern "C" {
const char* stand_in_names() {
  static std::string out;
  for (const auto& n : names)
    if (n.second.find("bsolve") != std::string::npos) out += name_of(n.first) + "\n";
  return out.c_str();
}
const char* stand_in_notes() { static std::string out; out.swap(notes); notes.clear(); return out.c_str(); }
void __cudaRegisterFunction(void** module, const char* host, char* fun, const char* device, int limit, uint3* tid,
                            uint3* bid, dim3* block, dim3* grid, int* warp) {
  names[host] = device;
  void* real = dlopen("libcudart.so.13", RTLD_LAZY | RTLD_NOLOAD);
  reinterpret_cast<decltype(&__cudaRegisterFunction)>(dlsym(real, "__cudaRegisterFunction"))(
      module, host, fun, device, limit, tid, bid, block, grid, warp);
}
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) {
    limits[f] = v;
    notes += "limit|" + name_of(f) + "|" + std::to_string(v) + "\n";
  }
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(&encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  return launched(f, c->gridDim, c->blockDim, c->dynamicSmemBytes, c->attrs[0].val.clusterDim.x);
}
cudaError_t __cudaGetKernel(void** kernel, const void* f) {
  *kernel = const_cast<void*>(f);
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(void* f, dim3 grid, dim3 block, void**, size_t shared, cudaStream_t) {
  return launched(f, grid, block, shared, 1);
}
}
"""

CHILD = r"""
import ctypes, json, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
fake.stand_in_notes.restype = fake.stand_in_names.restype = ctypes.c_char_p
sys.path.insert(0, sys.argv[2])
import dense_linear_solvers_gb300 as bs
from tests.test_delta_host import BACKWARD, FORWARD, PRODUCT, call
lib = bs.lib()
FAR = [k << 44 for k in range(1, 24)]  # operands too far apart to overlap, never dereferenced
TYPES = {"f32": (bs.BS_FP32, 4), "bf16": (bs.BS_BF16, 2), "f16": (bs.BS_FP16, 2)}

def notes():
    return [n.split("|") for n in fake.stand_in_notes().decode().splitlines()]

def delta(args, entry, kind, batch, length, hk, hv, dk, dv, pad, packed=False):
    # q, k, v and their gradients as windows of matrices with `pad` columns more
    dtype, size = TYPES[kind]
    ld, at = 2 * hk * dk + hv * dv + pad, pad // 2
    given = dict(args, dtype=dtype, heads_k=hk, heads_v=hv, dk=dk, dv=dv, batch=batch, rows=batch * length,
                 offsets=FAR[20] if packed else None)
    for n, names in enumerate((("q", "dq"), ("k", "d_k"), ("v", "d_v"))):
        for m, name in enumerate(names):
            if name in given:
                given[name] = FAR[m] + size * (at + n * hk * dk)
    for name, place in (("g", 2), ("beta", 3), ("h0", 4), ("o", 5), ("hT", 6), ("tape", 7), ("work", 8),
                        ("d_o", 9), ("dhT", 10), ("dg", 11), ("dbeta", 12), ("dh0", 13)):
        if name in given:
            given[name] = FAR[place]
    for name in ("ldq", "ldk", "ldv", "lddq", "lddk", "lddv"):
        if name in given:
            given[name] = ld
    for name, n in (("ldo", hv * dv), ("lddo", hv * dv), ("ldg", hv), ("ldbeta", hv), ("lddg", hv),
                    ("lddbeta", hv)):
        if name in given:
            given[name] = n
    given["work_bytes"] = 1 << 43
    return entry(*given.values())

def forward(*shape, **more):
    return delta(FORWARD, lib.bs_gdelta_batched, *shape, **more)

def backward(*shape, **more):
    return delta(BACKWARD, lib.bs_gdelta_backward_batched, *shape, **more)

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


def test_a_kernel_has_one_limit(stand_in):
    """A kernel's limit of shared memory belongs to the device, not to a host thread: a call that set its own
    size could lower it between another thread's setting and launch. Calls of every size set the same."""
    got = child(stand_in, """
out["status"] = []
for kind in TYPES:
    for dk in (64, 128):
        for hv in (1, 8, 40, 128, 300):
            for dv in (8, 24, 64, 120, 128, 256):
                out["status"] += [forward(kind, 1, 100, 1, hv, dk, dv, 0),
                                  backward(kind, 1, 100, 1, hv, dk, dv, 0)]
out["notes"] = notes()
""")
    assert set(got["status"]) == {0}
    limits = {}
    for what, name, value, *_ in got["notes"]:
        if what == "limit":
            limits.setdefault(name, set()).add(int(value))
    assert any("team_kernel" in n for n in limits) and any("chain_kernel" in n for n in limits)
    assert {n: v for n, v in limits.items() if len(v) > 1} == {}


def test_a_product_of_no_depth(stand_in):
    """Rows of no element may lie at any distance and on any address: nothing of them is read."""
    got = child(stand_in, """
f = lib.bs_gemm_q8
empty = dict(k=0, lda=1, ldw=1, ldsa=0, ldsw=0)
out["taken"] = [call(f, PRODUCT, **empty), call(f, PRODUCT, **empty, a=None, sa=None, w=None, sw=None),
                call(f, PRODUCT, **empty, a=FAR[0] + 3, sa=FAR[1] + 1, w=FAR[2] + 5, sw=FAR[3] + 2)]
out["kernels"] = [n[1].split("::")[-1].split("<")[0] for n in notes() if n[0] == "launch"]
out["refused"] = [call(f, PRODUCT, **empty, y=None), call(f, PRODUCT, lda=257), call(f, PRODUCT, ldw=257),
                  call(f, PRODUCT, k=1, lda=1, ldw=1, ldsa=1, ldsw=1)]
""")
    assert got["taken"] == [0] * 3 and got["refused"] == [1] * 4
    assert got["kernels"] == ["zero_kernel"] * 3


def test_every_compiled_chain_can_be_chosen(stand_in):
    got = child(stand_in, """
for kind in TYPES:
    for dk in (64, 128):
        for hv in (1, 40, 128, 300):
            for dv in (8, 24, 64, 128, 256):
                for pad in (0, 3):  # aligned rows and others
                    assert forward(kind, 1, 100, 1, hv, dk, dv, pad) == 0
                    assert backward(kind, 1, 100, 1, hv, dk, dv, pad) == 0
out["launched"] = sorted({n[1] for n in notes() if n[0] == "launch"})
out["compiled"] = fake.stand_in_names().decode().splitlines()
""")
    chains = {n for n in got["compiled"] if any(k in n for k in ("chain_kernel<", "team_kernel<", "back_kernel<"))}
    assert len(chains) == 2 * (12 + 12)  # teams and single warps: three types, two depths, aligned or not
    assert chains == {n for n in got["launched"] if n in chains}


def block_of(note):
    """How a chain's launch is made up, and 1 where its kernel takes aligned rows only."""
    name, threads = note[1], int(note[3])
    kernel, args = name.split("::")[-1][:-1].split("<")
    kind, deep, vec, last = args.split(", ")[-4:]
    if kernel.startswith("team"):
        loaders = 128 if deep == "64" or "bfloat16" in name else 256
        return f"{(threads - loaders) // 128} teams", vec == "true"
    return f"{threads // 32} warps", vec == "true"


def test_the_shapes_of_the_tests_reach_their_chains(stand_in):
    """Both passes take the form that the GPU's tests are there for, and all forms are among them, aligned and not."""
    got = child(stand_in, """
from tests.delta_forms import CHAINS, CUTS, PACKED
shapes = [(s, False) for s, _ in CHAINS] + [((kind, 5, CUTS[-1] // 5, *rest, 0), True) for kind, *rest in PACKED]
out["notes"] = []
for shape, packed in shapes:
    assert forward(*shape, packed=packed) == 0 and backward(*shape, packed=packed) == 0
    out["notes"].append([n for n in notes() if n[0] == "launch"])
""")
    forms = [f for _, f in CHAINS] + ["8 warps"] * len(PACKED)
    seen = set()
    for (shape, form, notes) in zip([s for s, _ in CHAINS] + PACKED, forms, got["notes"]):
        chains = [n for n in notes if any(k in n[1] for k in ("chain_kernel<", "team_kernel<", "back_kernel<"))]
        assert len(chains) == 2
        for n in chains:
            block, vec = block_of(n)
            assert block == form, (shape, block)
            seen.add((n[1].split("::")[-1], block))
    kernels = {k for k, _ in seen}
    for kind in ("float", "__half", "__nv_bfloat16"):
        for vec in ("true", "false"):
            for kernel in ("chain_kernel", "back_kernel"):
                assert f"{kernel}<{kind}, 128, {vec}, {2 if 'bf' in kind else 1}>" in kernels


def test_the_shapes_of_the_tests_reach_their_products(stand_in):
    got = child(stand_in, """
from tests.delta_forms import PRODUCTS
for (m, n, k, ld), _ in PRODUCTS:
    wide = -(-k // 16) * 16
    assert call(lib.bs_gemm_q8, PRODUCT, m=m, n=n, k=k, a=FAR[0], lda=wide, sa=FAR[1], ldsa=-(-k // 128), w=FAR[2],
                ldw=wide, sw=FAR[3], ldsw=-(-k // 128), y=FAR[4] + 2 * ld, ldy=n + 2 * ld) == 0
out["notes"] = [n for n in notes() if n[0] == "launch"]
""")
    assert len(got["notes"]) == len(PRODUCTS)
    for (shape, form), (_, name, _, _, _, cluster) in zip(PRODUCTS, got["notes"]):
        kernel, args = name.split("::")[-1][:-1].split("<")
        assert f"{kernel} {args.split(', ')[-1]} {cluster}" == form, (shape, name, cluster)
