"""The decode attention on a process's second device, on the CPU: attn.cu is compiled with the runtime's functions replaced
by ones that stand for two devices, keep each kernel's shared-memory limit for each device as CUDA does, and refuse a launch
above it. No kernel runs."""
import ctypes
import subprocess

import pytest

TWO_DEVICES = """
#include <cuda.h>
#include <cuda_runtime.h>
#include <map>
#include <utility>

static int current = 0, failing = 0, last_grid = 0;
static std::map<std::pair<int, const void*>, size_t> limits;
static cudaError_t fake_get_device(int* d) {
  *d = current;
  return cudaSuccess;
}
static cudaError_t fake_attribute(int* v, cudaDeviceAttr, int d) {
  *v = d == 0 ? 152 : 100;
  return cudaSuccess;
}
template <typename F>
cudaError_t fake_set(F* f, cudaFuncAttribute, int v) {
  if (failing > 0) {
    --failing;
    return cudaErrorInvalidValue;
  }
  limits[{current, reinterpret_cast<const void*>(f)}] = v;
  return cudaSuccess;
}
template <typename F>
cudaError_t fake_occupancy(int* n, F, int, size_t) {
  *n = 1;
  return cudaSuccess;
}
template <typename F, typename... A>
cudaError_t fake_launch(const cudaLaunchConfig_t* c, F* f, A&&...) {
  const auto at = limits.find({current, reinterpret_cast<const void*>(f)});
  if (c->dynamicSmemBytes > (at == limits.end() ? size_t{48} * 1024 : at->second)) return cudaErrorInvalidValue;
  if (c->dynamicSmemBytes > 0) last_grid = c->gridDim.x;
  return cudaSuccess;
}
static CUresult CUDAAPI fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
static cudaError_t fake_entry(const char*, void** p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
static cudaError_t fake_last() { return cudaSuccess; }
#define cudaGetDevice fake_get_device
#define cudaDeviceGetAttribute fake_attribute
#define cudaFuncSetAttribute fake_set
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor fake_occupancy
#define cudaLaunchKernelEx fake_launch
#define cudaGetDriverEntryPointByVersion fake_entry
#define cudaGetLastError fake_last
#include "attn.cu"
#define OUT extern "C" __attribute__((visibility("default")))
OUT void use_device(int d) { current = d; }
OUT void fail_next(int n) { failing = n; }
OUT int grid() { return last_grid; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import __graft_entry__
    b = __graft_entry__._builder()
    b.build()
    src = tmp_path_factory.mktemp("two_devices") / "two_devices.cu"
    src.write_text(TWO_DEVICES)
    so = str(src)[:-3] + ".so"
    flags = [f for f in b.NVCC_FLAGS if f not in ("-O3", "-lineinfo")]
    # the device code is not for running: intermediate code without optimisation, which builds in a third of the time
    subprocess.run([b._nvcc(), "-gencode", "arch=compute_103a,code=compute_103a", "-O0", "-Xcicc", "-O0", *flags, "-shared",
                    "-o", so, str(src)], check=True, capture_output=True)
    import kv_cache_pruning_gb300 as k
    lib = ctypes.CDLL(so)
    for fn in ("kvp_decode_attn_acc", "kvp_decode_attn", "kvp_decode_attn_two_tier"):
        getattr(lib, fn).restype, getattr(lib, fn).argtypes = k._SIGS[fn]
    return lib


def call(lib, fn, g, d):
    tables = (16, 16, 16, 16, 4, 16, 3)
    end = (0, 16, 1 << 40, None, None)
    if fn == "kvp_decode_attn_acc":
        return lib.kvp_decode_attn_acc(1, 2 * g, 2, d, *tables, 16, 16, 5, 0.0, 16, None, 16, 200, 100, 100, *end)
    if fn == "kvp_decode_attn":
        return lib.kvp_decode_attn(1, 2 * g, 2, d, *tables, 16, 5, 0.0, 16, *end)
    return lib.kvp_decode_attn_two_tier(1, 2 * g, 2, d, *tables, 16, 16, 16, 16, 4, 16, 3, 16, 5, 0.0, 16, *end)


@pytest.mark.parametrize("fn", ["kvp_decode_attn_acc", "kvp_decode_attn", "kvp_decode_attn_two_tier"])
@pytest.mark.parametrize("g", [1, 2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_every_device_gets_its_shared_memory_and_its_grid(lib, fn, g, d):
    from kv_cache_pruning_gb300 import KVP_ERR_CUDA, KVP_OK
    lib.use_device(0)
    lib.fail_next(1)
    assert call(lib, fn, g, d) == KVP_ERR_CUDA               # a failure is the call's own: the next one asks again
    lib.fail_next(0)
    for device, sms in ((0, 152), (1, 100), (0, 152), (63, 100), (64, 100), (64, 100), (1, 100)):
        lib.use_device(device)
        assert call(lib, fn, g, d) == KVP_OK, device
        assert lib.grid() == sms
