"""A bounded wait that gives up in the middle of a call: the kernel records KVP_ERR_TIMEOUT, drains what it has issued and
returns, and a call with state beside its outputs leaves that state alone. The kernels are compiled here once more with a
wait in place of the library's that waits as it does, and then one time in a call, of the test's choice, says that it
gave up: no barrier is left without its arrival, and nothing waits for longer than the library's limit."""
import concurrent.futures
import ctypes
import subprocess
import time

import pytest
import torch

from test_gpu_prompt import cache_of, i32, normal, qkv, status

pytestmark = pytest.mark.gpu

# The drains after a wait that gave up name no abort flag and no status word: they wait as they are.
GIVE_UP = """
#include "%(header)s"
namespace kvp {
__device__ int gives_up_at = -1, waits = 0;
KVP_DEV bool says_so(bool ok) {
  if ((threadIdx.x & 31) != 0) return ok;
  return atomicAdd(&waits, 1) != gives_up_at && ok;
}
KVP_DEV bool wait_or_give_up(uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity); }
KVP_DEV bool wait_or_give_up(uint64_t* bar, uint32_t parity, const volatile int* abort, const volatile int32_t* status,
                             uint64_t limit = kWaitLimitNs) {
  return says_so(mbar_wait(bar, parity, abort, status, limit));
}
%(quietly)s
}  // namespace kvp
#define mbar_wait wait_or_give_up
#include "%(source)s"
extern "C" __attribute__((visibility("default"))) int set_give_up(int at) {
  const int none = 0;
  int e = static_cast<int>(cudaDeviceSynchronize());
  e |= static_cast<int>(cudaMemcpyToSymbol(kvp::gives_up_at, &at, sizeof at));
  return e | static_cast<int>(cudaMemcpyToSymbol(kvp::waits, &none, sizeof none));
}
extern "C" __attribute__((visibility("default"))) int get_waits() {
  int n = -1;
  return cudaMemcpyFromSymbol(&n, kvp::waits, sizeof n) == cudaSuccess ? n : -1;
}
extern "C" __attribute__((visibility("default"))) int leave_error() {   // refused on the host: no such device
  return static_cast<int>(cudaSetDevice(1 << 20));
}
extern "C" __attribute__((visibility("default"))) int take_error() { return static_cast<int>(cudaGetLastError()); }
"""
QUIETLY = """
namespace {
KVP_DEV bool wait_quietly_or_give_up(uint64_t* bar, uint32_t parity, const volatile int* abort,
                                     const volatile int32_t* status) {
  return says_so(wait_quietly(bar, parity, abort, status));
}
}  // namespace
#define wait_quietly wait_quietly_or_give_up
"""
SOURCES = {"attn": ("kvp_common.cuh", ""), "prompt": ("prompt.cuh", QUIETLY), "prompt_weights": ("prompt.cuh", QUIETLY)}


@pytest.fixture(scope="module")
def libs(kvp, tmp_path_factory):
    import __graft_entry__
    b = __graft_entry__._builder()
    at = tmp_path_factory.mktemp("give_up")

    def build(name):
        header, quietly = SOURCES[name]
        src = at / f"{name}_beside.cu"
        src.write_text(GIVE_UP % dict(header=header, quietly=quietly, source=name + ".cu"))
        so = str(src)[:-3] + ".so"
        subprocess.run([b._nvcc(), *b.ARCH, *b.NVCC_FLAGS, "-shared", "-o", so, str(src)], check=True, capture_output=True)
        return so

    with concurrent.futures.ThreadPoolExecutor() as ex:
        built = dict(zip(SOURCES, ex.map(build, SOURCES)))
    libs = {name: ctypes.CDLL(so) for name, so in built.items()}
    for name, fns in (("attn", ["kvp_decode_attn_acc"]), ("prompt", ["kvp_prompt_attn"]),
                      ("prompt_weights", ["kvp_prompt_weights"])):
        for fn in fns:
            getattr(libs[name], fn).restype, getattr(libs[name], fn).argtypes = kvp._SIGS[fn]
    return libs


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("g, counts", [(1, [[5000, 40]]), (2, [[3000, 3000]]), (4, [[5000, 40]]), (8, [[700, 9000]])])
def test_decode_sums_stay_where_a_wait_gave_up(kvp, libs, g, counts):
    lib, h, d, t = libs["attn"], 2, 128, 9100
    width = (max(counts[0]) + 15) // 16
    cache = cache_of(kvp, 3, counts, width, d, h, t)
    q, first = normal(5, 1, h * g, d), torch.rand(1, h, t, device="cuda")
    n = kvp.kvp_decode_attn_acc_workspace_bytes(1, h * g, h, d, width)
    ws, out, acc, st = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.empty(1, h * g, d, device="cuda"), first.clone(), status()
    want, want_acc = torch.empty_like(out), first.clone()
    kvp.kvp_decode_attn_acc(q, cache, t - 1, want_acc, out=want, workspace=torch.zeros_like(ws), status=st)
    assert int(st) == 0

    def call(at, with_status=True):
        st.zero_()
        assert lib.set_give_up(at) == 0
        assert lib.kvp_decode_attn_acc(
            1, h * g, h, d, q.data_ptr(), cache.k_pool.data_ptr(), cache.v_pool.data_ptr(), cache.expire_pool.data_ptr(),
            cache.n_pages_cap, cache.page_table.data_ptr(), width, cache.remap.data_ptr(), cache.count.data_ptr(), t - 1,
            0.0, out.data_ptr(), None, acc.data_ptr(), acc.stride(0), acc.stride(1), t, 0, ws.data_ptr(), n,
            st.data_ptr() if with_status else None, stream()) == kvp.KVP_OK
        torch.cuda.synchronize()
        return int(st)

    assert call(-1) == 0 and torch.equal(acc, want_acc)      # (one addition a sum: the same bits)
    waits = lib.get_waits()
    assert waits > 20
    for at in (0, waits // 2, waits - 1):
        for with_status in (True, False):
            ws.zero_()
            acc.copy_(first)
            assert call(-1) == 0 and torch.equal(acc, want_acc)   # leaves the logits and sums of a finished step behind
            acc.copy_(first)
            code = call(at, with_status)
            assert code == (kvp.KVP_ERR_TIMEOUT if with_status else 0) and torch.equal(acc, first)
            # the workspace is to be zeroed before its next use; until then nothing is added, and the call says so
            assert call(-1) == kvp.KVP_ERR_TIMEOUT and torch.equal(acc, first)
    ws.zero_()
    assert call(-1) == 0 and torch.equal(acc, want_acc) and torch.equal(out, want)


@pytest.mark.parametrize("h, g, d, lens", [(2, 4, 128, [700, 900, 30]), (2, 3, 128, [900, 130, 700]), (2, 3, 64, [900, 130, 700]),
                                           (2, 2, 64, [300, 1, 900]), (1, 1, 128, [300]), (1, 2, 64, [500])])
def test_prompt_calls_end_where_a_wait_gave_up(kvp, libs, h, g, d, lens):
    """Each call returns and says so (or is right: a wait at a CTA's end, for what is on its way to the CTA itself), and the
    next one is right. One tile an item and two, of two heads and of two tiles."""
    lens = lens * (30 if len(lens) > 1 else 1)
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    n, hq, start = start[-1], h * g, i32(start)
    q, k, v = (x.contiguous() for x in qkv(6, n, hq, h, d))
    want, want_lse = torch.empty_like(q), torch.empty(hq, n, device="cuda")
    kvp.kvp_prompt_attn(q, k, v, start, out=want, lse=want_lse)
    st, out, lse = status(), torch.empty_like(q), torch.empty_like(want_lse)

    def attend(at):
        st.zero_()
        assert libs["prompt"].set_give_up(at) == 0
        assert libs["prompt"].kvp_prompt_attn(
            len(lens), n, hq, h, d, q.data_ptr(), *q.stride()[:2], k.data_ptr(), *k.stride()[:2], v.data_ptr(),
            *v.stride()[:2], start.data_ptr(), None, 0.0, out.data_ptr(), *out.stride()[:2], lse.data_ptr(), st.data_ptr(),
            stream()) == kvp.KVP_OK
        torch.cuda.synchronize()
        return int(st)

    def weigh(at, n_last, acc):
        st.zero_()
        assert libs["prompt_weights"].set_give_up(at) == 0
        assert libs["prompt_weights"].kvp_prompt_weights(
            len(lens), n, hq, h, d, q.data_ptr(), *q.stride()[:2], k.data_ptr(), *k.stride()[:2], start.data_ptr(), None,
            want_lse.data_ptr(), 0.0, n_last, acc.data_ptr(), -1, *acc.stride(), 0, st.data_ptr(), stream()) == kvp.KVP_OK
        torch.cuda.synchronize()
        return int(st)

    assert attend(-1) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    waits = libs["prompt"].get_waits()
    assert waits > 20
    for at in [0, 1, 5, waits // 3, waits // 2, 2 * waits // 3, waits - 2, waits - 1]:
        before = time.monotonic()
        code = attend(at)
        assert time.monotonic() - before < 1.5
        assert code == kvp.KVP_ERR_TIMEOUT or at > 0 and code == 0 and torch.equal(out, want) and torch.equal(lse, want_lse), at
    assert attend(-1) == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)
    for n_last in (0, 40):
        want_acc, acc = kvp.kvp_prompt_weights(q, k, start, want_lse, n_last=n_last), torch.zeros(n, h, device="cuda")
        assert weigh(-1, n_last, acc) == 0 and torch.equal(acc, want_acc)
        waits = libs["prompt_weights"].get_waits()
        for at in [0, 1, 5, waits // 3, waits // 2, 2 * waits // 3, waits - 2, waits - 1]:
            before = time.monotonic()
            code = weigh(at, n_last, acc.zero_())
            assert time.monotonic() - before < 1.5                # one wait gave up: no other runs to the limit of two seconds
            assert code == kvp.KVP_ERR_TIMEOUT or at > 0 and code == 0 and torch.equal(acc, want_acc), at
        assert weigh(-1, n_last, acc) == 0 and torch.equal(acc, want_acc)


# ---------------------------------------------------------------------------- a caller's pending error

@pytest.mark.parametrize("g", [1, 2, 4, 8])
def test_a_pending_error_stays_the_callers(kvp, libs, g):
    """An error of the runtime's that the caller has left pending is neither taken away nor reported by a call: reported
    between the attention and the kernel that adds, it left the sums out."""
    lib, h, d, t = libs["attn"], 2, 64, 400
    cache = cache_of(kvp, 3, [[300, 40]], 20, d, h, t)
    q, acc, want = normal(5, 1, h * g, d), torch.zeros(1, h, t, device="cuda"), torch.zeros(1, h, t, device="cuda")
    st, out = status(), torch.empty(1, h * g, d, device="cuda")
    n = kvp.kvp_decode_attn_acc_workspace_bytes(1, h * g, h, d, 20)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    kvp.kvp_decode_attn_acc(q, cache, t - 1, want)
    assert lib.set_give_up(-1) == 0 and lib.take_error() == 0
    for turn in range(2):                                    # (the runtime drops it itself where it first loads a kernel)
        acc.zero_()
        left = lib.leave_error()
        assert left != 0
        code = lib.kvp_decode_attn_acc(
            1, h * g, h, d, q.data_ptr(), cache.k_pool.data_ptr(), cache.v_pool.data_ptr(), cache.expire_pool.data_ptr(),
            cache.n_pages_cap, cache.page_table.data_ptr(), 20, cache.remap.data_ptr(), cache.count.data_ptr(), t - 1, 0.0,
            out.data_ptr(), None, acc.data_ptr(), acc.stride(0), acc.stride(1), t, 0, ws.data_ptr(), n, st.data_ptr(),
            stream())
        pending = lib.take_error()
        torch.cuda.synchronize()
        assert code == kvp.KVP_OK and int(st) == 0 and torch.equal(acc, want)
        assert turn == 0 or pending == left
