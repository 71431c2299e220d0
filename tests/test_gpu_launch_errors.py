"""A caller's own pending CUDA error is the caller's: a write that is launched returns KVP_OK and leaves that error to be
read. The library has a CUDA runtime of its own, so the write is compiled here once more with two functions beside it
that leave such an error and read it."""
import ctypes
import os
import subprocess

import pytest
import torch

import kvp_synth as syn
from helpers import dev_bf16, status_word

pytestmark = pytest.mark.gpu

BESIDE = """
#include "block8.cu"
#define OUT extern "C" __attribute__((visibility("default")))
OUT int leave_error() { return static_cast<int>(cudaSetDevice(1 << 20)); }   // refused on the host: no such device
OUT int take_error() { return static_cast<int>(cudaGetLastError()); }
"""


@pytest.fixture(scope="module")
def beside(kvp, tmp_path_factory):
    import __graft_entry__
    b = __graft_entry__._builder()
    src = tmp_path_factory.mktemp("beside") / "beside.cu"
    src.write_text(BESIDE)
    so = str(src)[:-3] + ".so"
    subprocess.run([b._nvcc(), *b.ARCH, *b.NVCC_FLAGS, "-shared", "-o", so, str(src)], check=True, capture_output=True)
    lib = ctypes.CDLL(so)
    lib.kvp_compact_block8.restype, lib.kvp_compact_block8.argtypes = kvp._SIGS["kvp_compact_block8"]
    return lib


# one launch, the passes, the passes with zeroed counts, the passes with the page-base pass
@pytest.mark.parametrize("B,T", [(2, 100), (2, 1100), (2, 4200), (600, 20)])
def test_a_pending_error_stays_the_callers(kvp, beside, B, T):
    H, d = 2, 64
    width = (T + 15) // 16
    k = dev_bf16(syn.normal_bf16(701, 1, (B, T, H, d)))
    flag = torch.full((B, H, T), -1, dtype=torch.int32, device="cuda")
    want = kvp.Block8PagedKV.allocate(B, H, d, B * H * width, width)
    got = kvp.Block8PagedKV.allocate(B, H, d, B * H * width, width)
    st = status_word()
    kvp.kvp_compact_block8(k, k, T - 1, 0, want, mode=1, flag_step=flag, status=st)
    n = kvp.kvp_compact_block8_workspace_bytes(B, H, T, B * H * width)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert beside.take_error() == 0
    left = beside.leave_error()
    assert left != 0
    code = beside.kvp_compact_block8(
        0, 1, B, H, d, T, k.data_ptr(), k.data_ptr(), *k.stride()[:3], None, None, flag.data_ptr(), 128, 0, T - 1, 0,
        got.kq_pool.data_ptr(), got.vq_pool.data_ptr(), got.scale_pool.data_ptr(), got.expire_pool.data_ptr(),
        B * H * width, got.page_table.data_ptr(), width, got.remap.data_ptr(), got.count.data_ptr(), ws.data_ptr(), n,
        st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    pending = beside.take_error()
    torch.cuda.synchronize()
    assert code == kvp.KVP_OK and pending == left and st.item() == 0
    for name in ("kq_pool", "vq_pool", "scale_pool", "expire_pool", "page_table", "remap", "count"):
        assert torch.equal(getattr(want, name), getattr(got, name)), name
