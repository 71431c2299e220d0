"""Python binding of libkvp (KV-cache pruning at decode time, sm_103a).

Each function here has the name of the C entry point it calls (see
include/kvp.h) and only marshals arguments: torch tensors are checked for
dtype, device and contiguity, their device pointers and sizes are passed on,
and a non-OK status raises KvpError. Every step of the path runs in the
library's CUDA kernels; there is no other implementation to fall back on, so
importing this package fails loudly when libkvp.so has not been built.

PyTorch is used for device memory and streams only: calls are enqueued on
torch's current CUDA stream unless a stream is passed.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvp.so")

KVP_OK = 0
KVP_ERR_INVALID = 1
KVP_ERR_ALIGN = 2
KVP_ERR_CAPACITY = 3
KVP_ERR_CUDA = 4
KVP_ERR_TIMEOUT = 5
KVP_ERR_UNSUPPORTED = 6
KVP_ERR_WORKSPACE = 7
KVP_ERR_BOUNDS = 8

KVP_SCORER_LINEAR = 0
KVP_SCORER_MLP = 1
KVP_SCORER_LINEAR_SPLIT = 2
KVP_MASK_KVZAP = 0
KVP_MASK_DMS = 1
KVP_BLOCK8_E4M3 = 0
KVP_BLOCK8_INT8 = 1
PAGE = 16
WINDOW = 128
EXPIRE_NEVER = 2**31 - 1
KVP_MLA_LATENT_DIM = 512
KVP_MLA_ROPE_DIM = 64
LATENT_ROW = KVP_MLA_LATENT_DIM + KVP_MLA_ROPE_DIM


class KvpError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn}: {status_string(code)} (status {code})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkvp.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    return ctypes.CDLL(LIB_PATH)


_lib = _load()

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_S = ctypes.c_size_t
_F = ctypes.c_float

_SIGS = {
    "kvp_status_string": (ctypes.c_char_p, [_I]),
    "kvp_version": (_I, []),
    "kvp_score_workspace_bytes": (_S, [_I, _L, _I, _I, _I]),
    "kvp_score_split_weight_bytes": (_S, [_I, _I]),
    "kvp_score_split_weight": (_I, [_I, _I, _P, _P, _S, _P]),
    "kvp_score": (_I, [_I, _L, _I, _I, _I, _P, _L, _P, _P, _P, _P, _P, _P, _S, _P, _P]),
    "kvp_mask": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "kvp_threshold_workspace_bytes": (_S, [_I, _I]),
    "kvp_threshold": (_I, [_I, _I, _I, _P, ctypes.c_double, _P, _P, _S, _P]),
    "kvp_compact_workspace_bytes": (_S, [_I, _I, _I]),
    "kvp_compact": (_I, [_I, _I, _I, _I, _P, _P, _L, _L, _L, _P, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P,
                         _P, _S, _P, _P]),
    "kvp_compact_masked": (_I, [_I, _I, _I, _I, _I, _P, _P, _L, _L, _L, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P,
                                _I, _P, _I, _P, _P, _P, _S, _P, _P]),
    "kvp_compact_quant": (_I, [_I, _I, _I, _I, _I, _P, _P, _L, _L, _L, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P,
                               _I, _P, _I, _P, _P, _P, _S, _P, _P]),
    "kvp_compact_noalloc": (_I, [_I, _I, _I, _I, _P, _P, _L, _L, _L, _P, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P,
                                 _P, _P]),
    "kvp_compact_paged_workspace_bytes": (_S, [_I, _I, _I]),
    "kvp_compact_paged": (_I, [_I, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _P, _P, _P, _I, _P, _I,
                               _P, _P, _P, _S, _P, _P]),
    "kvp_append": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P,
                        _P, _P]),
    "kvp_append_devpos": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P,
                               _P, _P]),
    "kvp_append_quant": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _I, _P, _I, _P, _P,
                              _P, _P]),
    "kvp_decode_attn_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "kvp_decode_attn": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _I, _F, _P, _I, _P, _S, _P, _P]),
    "kvp_decode_attn_devpos": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _P, _F, _P, _I, _P, _S, _P,
                                    _P]),
    "kvp_decode_attn_lse": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _I, _F, _P, _P, _I, _P, _S, _P,
                                 _P]),
    "kvp_attn_merge": (_I, [_I, _L, _I, _P, _P, _P, _P, _P]),
    "kvp_decode_attn_two_tier": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _P, _I, _P, _I, _P,
                                      _I, _F, _P, _I, _P, _S, _P, _P]),
    "kvp_compact_latent": (_I, [_I, _I, _I, _I, _P, _L, _L, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _I, _P, _P,
                                _P, _S, _P, _P]),
    "kvp_compact_latent_paged": (_I, [_I, _I, _P, _P, _I, _P, _I, _P, _P, _I, _I, _P, _P, _I, _P, _I, _P, _P, _P,
                                      _S, _P, _P]),
    "kvp_append_latent": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _P, _P, _I, _P, _I, _P, _P, _P, _P]),
    "kvp_selftest_wait": (_I, [ctypes.c_uint64, _P, _P, _P]),
    "kvp_compact_block8_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "kvp_compact_block8": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _L, _L, _L, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P,
                                _P, _I, _P, _I, _P, _P, _P, _S, _P, _P]),
    "kvp_append_block8": (_I, [_I, _I, _I, _I, _I, _I, _P, _P, _L, _L, _L, _L, _P, _P, _P, _I, _I, _P, _P, _P, _P, _I,
                               _P, _I, _P, _P, _P, _P]),
    "kvp_append_block8_devpos": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _L, _L, _L, _L, _P, _P, _P, _I, _I, _P, _P, _P,
                                      _P, _I, _P, _I, _P, _P, _P, _P]),
    "kvp_read_block8": (_I, [_I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _L, _L, _L, _P, _P]),
    "kvp_decode_attn_block8_workspace_bytes": (_S, [_I, _I, _I, _I]),
    "kvp_decode_attn_block8": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _I, _P, _I, _F, _P, _P, _I, _P, _S,
                                    _P, _P]),
    "kvp_decode_attn_block8_devpos": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _F, _P, _P, _I,
                                           _P, _S, _P, _P]),
    "kvp_rope_turns": (_I, [_I, _P, _P]),
    "kvp_qk_norm_rope": (_I, [_L, _I, _I, _I, _I, _I, _P, _L, _L, _P, _L, _L, _P, _P, _P, _P, _F, _P, _L, _L, _P, _L, _L,
                              _P]),
    "kvp_prompt_attn": (_I, [_I, _L, _I, _I, _I, _P, _L, _L, _P, _L, _L, _P, _L, _L, _P, _P, _F, _P, _L, _L, _P, _P, _P]),
    "kvp_prompt_weights": (_I, [_I, _L, _I, _I, _I, _P, _L, _L, _P, _L, _L, _P, _P, _P, _F, _I, _P, _L, _L, _L, _I, _P,
                                _P]),
    "kvp_decode_attn_acc_workspace_bytes": (_S, [_I, _I, _I, _I, _I]),
    "kvp_decode_attn_acc": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _P, _I, _F, _P, _P, _P, _L, _L, _I, _I,
                                 _P, _S, _P, _P]),
    "kvp_decode_attn_acc_devpos": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _I, _P, _P, _P, _F, _P, _P, _P, _L, _L,
                                        _I, _I, _P, _S, _P, _P]),
    "kvp_evict": (_I, [_I, _I, _I, _P, _L, _L, _L, _I, _I, _I, _P, _P, _P]),
    "kvp_evict_paged": (_I, [_I, _I, _P, _L, _L, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _P, _P, _P]),
    "kvp_evict_paged_devpos": (_I, [_I, _I, _P, _L, _L, _I, _P, _I, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P]),
    "kvp_decode_attn_mla_workspace_bytes": (_S, [_I, _I, _I]),
    "kvp_decode_attn_mla": (_I, [_I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _P, _I, _F, _P, _I, _P, _S, _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def library():
    """The loaded ctypes handle of libkvp.so."""
    return _lib


def status_string(code: int) -> str:
    return _lib.kvp_status_string(int(code)).decode()


def version() -> int:
    return _lib.kvp_version()


# --------------------------------------------------------------------------- marshalling helpers

def _ptr(t, dtype=None, name="tensor", optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, code: int):
    if code != KVP_OK:
        raise KvpError(fn, code)


def _ws(nbytes: int, device, workspace=None):
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------- score

def kvp_score_workspace_bytes(scorer, n_tok, d_model, n_kv_heads, hidden=0) -> int:
    return _lib.kvp_score_workspace_bytes(scorer, n_tok, d_model, n_kv_heads, hidden)


def kvp_score_split_weight_bytes(d_model, n_kv_heads) -> int:
    return _lib.kvp_score_split_weight_bytes(d_model, n_kv_heads)


def kvp_score_split_weight(w, *, out=None, stream=None):
    """The KVzap-Linear weight w fp32 [H, D] as the scorer's bf16 hi/lo operand (rows 2h, 2h+1), for
    kvp_score(..., scorer=KVP_SCORER_LINEAR_SPLIT, n_kv_heads=H)."""
    H, D = w.shape
    nbytes = kvp_score_split_weight_bytes(D, H)
    if out is None:
        out = torch.empty((nbytes // (2 * D), D), dtype=torch.bfloat16, device=w.device)
    code = _lib.kvp_score_split_weight(D, H, _ptr(w, torch.float32, "w"), _ptr(out, torch.bfloat16, "out"),
                                       out.numel() * out.element_size(), _stream(stream))
    _check("kvp_score_split_weight", code)
    return out


def kvp_score(x, w, b=None, w2=None, b2=None, *, scorer=KVP_SCORER_LINEAR, n_kv_heads=None, out=None,
              workspace=None, status=None, stream=None):
    """scores[n_tok, H] from hidden states x[n_tok, D] (bf16).

    LINEAR: w fp32 [H, D], b fp32 [H] or None.
    LINEAR_SPLIT: w the bf16 operand from kvp_score_split_weight, n_kv_heads = H, b as for LINEAR.
    MLP:    w bf16 W1 [hidden, D], b fp32 b1 [hidden] or None, w2 bf16 [H, hidden], b2 fp32 [H] or None.
    """
    if x.dim() != 2:
        raise ValueError("x must be [n_tok, D]")
    n_tok, D = x.shape
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    if scorer == KVP_SCORER_LINEAR:
        H, hidden = w.shape[0], 0
        wp = _ptr(w, torch.float32, "w")
    elif scorer == KVP_SCORER_LINEAR_SPLIT:
        if n_kv_heads is None:
            raise ValueError("LINEAR_SPLIT needs n_kv_heads")
        H, hidden = int(n_kv_heads), 0
        wp = _ptr(w, torch.bfloat16, "w_split")
    else:
        hidden, H = w.shape[0], w2.shape[0]
        wp = _ptr(w, torch.bfloat16, "w1")
    if out is None:
        out = torch.empty((n_tok, H), dtype=torch.float32, device=x.device)
    need = kvp_score_workspace_bytes(scorer, n_tok, D, H, hidden)
    ws = _ws(need, x.device, workspace)
    code = _lib.kvp_score(scorer, n_tok, D, H, hidden, x.data_ptr(), x.stride(0), wp,
                          _ptr(b, torch.float32, "b", True),
                          _ptr(w2, torch.bfloat16, "w2", True), _ptr(b2, torch.float32, "b2", True),
                          _ptr(out, torch.float32, "out"), ws.data_ptr(), ws.numel() * ws.element_size(),
                          _ptr(status, torch.int32, "status", True), _stream(stream))
    _check("kvp_score", code)
    return out


# --------------------------------------------------------------------------- mask

def kvp_mask(*, mode, batch, n_kv_heads, n_pos, now, scores=None, tau=None, flag_step=None, window=WINDOW,
             delay=0, pos0=0, expire=None, keep_bits=None, count=None, want_bits=True, stream=None):
    """expire [B, H, n_pos] (+ keep_bits, count) from KVzap scores [B, n_pos, H] and tau [B, H], or from
    DMS flag steps [B, H, n_pos]."""
    dev = (scores if scores is not None else flag_step).device
    if expire is None:
        expire = torch.empty((batch, n_kv_heads, n_pos), dtype=torch.int32, device=dev)
    if want_bits and keep_bits is None:
        keep_bits = torch.empty((batch, n_kv_heads, (n_pos + 31) // 32), dtype=torch.int32, device=dev)
    if count is None:
        count = torch.empty((batch, n_kv_heads), dtype=torch.int32, device=dev)
    code = _lib.kvp_mask(mode, batch, n_kv_heads, n_pos, pos0, _ptr(scores, torch.float32, "scores", True),
                         _ptr(tau, torch.float32, "tau", True), _ptr(flag_step, torch.int32, "flag_step", True),
                         window, delay, now, _ptr(expire, torch.int32, "expire"),
                         _ptr(keep_bits, torch.int32, "keep_bits", True), _ptr(count, torch.int32, "count"),
                         _stream(stream))
    _check("kvp_mask", code)
    return expire, keep_bits, count


# --------------------------------------------------------------------------- paged cache

@dataclass
class PagedKV:
    """Device buffers of one compacted cache (allocated with torch)."""
    k_pool: torch.Tensor        # bf16 [n_pages_cap, 16, d]
    v_pool: torch.Tensor        # bf16 [n_pages_cap, 16, d]
    expire_pool: torch.Tensor   # int32 [n_pages_cap, 16]
    page_table: torch.Tensor    # int32 [B, H, max_pages]
    remap: torch.Tensor         # int32 [B, H, max_pages * 16]
    count: torch.Tensor         # int32 [B, H]

    @staticmethod
    def allocate(batch, n_kv_heads, head_dim, n_pages_cap, max_pages, device="cuda"):
        return PagedKV(
            torch.zeros((n_pages_cap, PAGE, head_dim), dtype=torch.bfloat16, device=device),
            torch.zeros((n_pages_cap, PAGE, head_dim), dtype=torch.bfloat16, device=device),
            torch.zeros((n_pages_cap, PAGE), dtype=torch.int32, device=device),
            torch.full((batch, n_kv_heads, max_pages), -1, dtype=torch.int32, device=device),
            torch.full((batch, n_kv_heads, max_pages * PAGE), -1, dtype=torch.int32, device=device),
            torch.zeros((batch, n_kv_heads), dtype=torch.int32, device=device),
        )

    @property
    def n_pages_cap(self):
        return self.k_pool.shape[0]

    @property
    def max_pages(self):
        return self.page_table.shape[2]

    @property
    def head_dim(self):
        return self.k_pool.shape[2]


@dataclass
class QuantPagedKV:
    """Device buffers of the fp8 tier (quantize instead of drop)."""
    kq_pool: torch.Tensor       # uint8 [n_pages_cap, 16, d] E4M3 codes of K rows
    vq_pool: torch.Tensor       # uint8 [n_pages_cap, 16, d] E4M3 codes of V rows
    meta_pool: torch.Tensor     # int32 [n_pages_cap, 3, 16]: start step, K scale, V scale (fp32 bits)
    page_table: torch.Tensor    # int32 [B, H, max_pages]
    remap: torch.Tensor         # int32 [B, H, max_pages * 16]
    count: torch.Tensor         # int32 [B, H]

    @staticmethod
    def allocate(batch, n_kv_heads, head_dim, n_pages_cap, max_pages, device="cuda"):
        return QuantPagedKV(
            torch.zeros((n_pages_cap, PAGE, head_dim), dtype=torch.uint8, device=device),
            torch.zeros((n_pages_cap, PAGE, head_dim), dtype=torch.uint8, device=device),
            torch.zeros((n_pages_cap, 3, PAGE), dtype=torch.int32, device=device),
            torch.full((batch, n_kv_heads, max_pages), -1, dtype=torch.int32, device=device),
            torch.full((batch, n_kv_heads, max_pages * PAGE), -1, dtype=torch.int32, device=device),
            torch.zeros((batch, n_kv_heads), dtype=torch.int32, device=device),
        )

    @property
    def n_pages_cap(self):
        return self.kq_pool.shape[0]

    @property
    def max_pages(self):
        return self.page_table.shape[2]

    @property
    def head_dim(self):
        return self.kq_pool.shape[2]

    @property
    def start_pool(self):
        return self.meta_pool[:, 0, :]

    @property
    def kscale(self):
        return self.meta_pool[:, 1, :].view(torch.float32)

    @property
    def vscale(self):
        return self.meta_pool[:, 2, :].view(torch.float32)


def kvp_threshold_workspace_bytes(batch, n_kv_heads) -> int:
    return _lib.kvp_threshold_workspace_bytes(batch, n_kv_heads)


def kvp_threshold(scores, q, *, out=None, workspace=None, stream=None):
    """Per-(b, h) threshold: the rank floor(q * (T - 1)) score of scores
    [B, T, H] along T (NaN ranked last) -> tau fp32 [B, H]."""
    if scores.dim() != 3:
        raise ValueError("scores must be [B, T, H]")
    B, T, H = scores.shape
    dev = scores.device
    tau = out if out is not None else torch.empty(B, H, dtype=torch.float32, device=dev)
    if tau.numel() != B * H:
        raise ValueError("out must hold B*H values")
    ws = _ws(kvp_threshold_workspace_bytes(B, H), dev, workspace)
    code = _lib.kvp_threshold(B, H, T, _ptr(scores, torch.float32, "scores"), float(q),
                              _ptr(tau, torch.float32, "out"), ws.data_ptr(), ws.numel() * ws.element_size(),
                              _stream(stream))
    _check("kvp_threshold", code)
    return tau


def kvp_compact_workspace_bytes(batch, n_kv_heads, n_pos) -> int:
    return _lib.kvp_compact_workspace_bytes(batch, n_kv_heads, n_pos)


def kvp_compact(k, v, expire, now, reserve, dst: PagedKV, *, status, workspace=None, stream=None):
    """Dense K, V [B, T, H, d] (any strides with d contiguous) + expire [B, H, T] -> dst."""
    B, T, H, d = k.shape
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v need identical strides with the head_dim axis contiguous")
    need = kvp_compact_workspace_bytes(B, H, T)
    ws = _ws(need, k.device, workspace)
    for t, nm in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{nm} must be a CUDA bf16 tensor")
    code = _lib.kvp_compact(B, H, d, T, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                            _ptr(expire, torch.int32, "expire"), now, reserve,
                            _ptr(dst.k_pool, torch.bfloat16), _ptr(dst.v_pool, torch.bfloat16),
                            _ptr(dst.expire_pool, torch.int32), dst.n_pages_cap,
                            _ptr(dst.page_table, torch.int32), dst.max_pages, _ptr(dst.remap, torch.int32),
                            _ptr(dst.count, torch.int32), ws.data_ptr(), ws.numel() * ws.element_size(),
                            _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_compact", code)
    return dst


def kvp_compact_noalloc(k, v, expire, now, reserve, dst: PagedKV, *, status, stream=None):
    """kvp_compact with its scratch in the library's fixed device array: allocates nothing (not even through
    torch). The first call on a device looks the array's address up, so make it before any stream capture; calls
    that overlap on the GPU race on the array."""
    B, T, H, d = k.shape
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v need identical strides with the head_dim axis contiguous")
    for t, nm in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{nm} must be a CUDA bf16 tensor")
    code = _lib.kvp_compact_noalloc(B, H, d, T, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                                    _ptr(expire, torch.int32, "expire"), now, reserve,
                                    _ptr(dst.k_pool, torch.bfloat16), _ptr(dst.v_pool, torch.bfloat16),
                                    _ptr(dst.expire_pool, torch.int32), dst.n_pages_cap,
                                    _ptr(dst.page_table, torch.int32), dst.max_pages, _ptr(dst.remap, torch.int32),
                                    _ptr(dst.count, torch.int32), _ptr(status, torch.int32, "status"),
                                    _stream(stream))
    _check("kvp_compact_noalloc", code)
    return dst


def kvp_compact_masked(k, v, now, reserve, dst: PagedKV, *, mode, scores=None, tau=None, flag_step=None,
                       window=WINDOW, delay=0, status, workspace=None, stream=None):
    """Dense K, V [B, T, H, d] with the mask applied on the fly: KVzap scores
    [B*T, H] (or [B, T, H]) + tau [B, H], or DMS flag_step [B, H, T] -> dst.
    Same result as kvp_mask (pos0 = 0) followed by kvp_compact."""
    B, T, H, d = k.shape
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v need identical strides with the head_dim axis contiguous")
    for t, nm in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{nm} must be a CUDA bf16 tensor")
    if scores is not None and scores.numel() != B * T * H:
        raise ValueError("scores must hold B*T*H values")
    if flag_step is not None and flag_step.numel() != B * H * T:
        raise ValueError("flag_step must hold B*H*T values")
    if tau is not None and tau.numel() != B * H:
        raise ValueError("tau must hold B*H values")
    need = kvp_compact_workspace_bytes(B, H, T)
    ws = _ws(need, k.device, workspace)
    code = _lib.kvp_compact_masked(mode, B, H, d, T, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                                   k.stride(2), _ptr(scores, torch.float32, "scores", True),
                                   _ptr(tau, torch.float32, "tau", True),
                                   _ptr(flag_step, torch.int32, "flag_step", True), window, delay, now, reserve,
                                   _ptr(dst.k_pool, torch.bfloat16), _ptr(dst.v_pool, torch.bfloat16),
                                   _ptr(dst.expire_pool, torch.int32), dst.n_pages_cap,
                                   _ptr(dst.page_table, torch.int32), dst.max_pages, _ptr(dst.remap, torch.int32),
                                   _ptr(dst.count, torch.int32), ws.data_ptr(), ws.numel() * ws.element_size(),
                                   _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_compact_masked", code)
    return dst


def kvp_compact_quant(k, v, scores, tau, tau_q, dst: QuantPagedKV, *, mode=KVP_MASK_KVZAP, flag_step=None, delay=0,
                      reserve=0, window=WINDOW, status, workspace=None, stream=None):
    """Dense K, V [B, T, H, d] -> the fp8 tier: entries with tau_q <= score < tau (scores [B*T, H] or
    [B, T, H]; tau, tau_q [B, H]), or with mode KVP_MASK_DMS the flagged entries (flag_step [B, H, T];
    scores, tau, tau_q None), as E4M3 codes with a per-row scale, visible from the step their bf16 copy
    is gone."""
    B, T, H, d = k.shape
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v need identical strides with the head_dim axis contiguous")
    for t, nm in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{nm} must be a CUDA bf16 tensor")
    if mode == KVP_MASK_KVZAP and (scores.numel() != B * T * H or tau.numel() != B * H or tau_q.numel() != B * H):
        raise ValueError("scores must hold B*T*H values, tau and tau_q B*H")
    if mode == KVP_MASK_DMS and flag_step.numel() != B * H * T:
        raise ValueError("flag_step must hold B*H*T values")
    need = kvp_compact_workspace_bytes(B, H, T)
    ws = _ws(need, k.device, workspace)
    code = _lib.kvp_compact_quant(mode, B, H, d, T, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                                  k.stride(2), _ptr(scores, torch.float32, "scores", True),
                                  _ptr(tau, torch.float32, "tau", True), _ptr(tau_q, torch.float32, "tau_q", True),
                                  _ptr(flag_step, torch.int32, "flag_step", True), window, delay, reserve,
                                  _ptr(dst.kq_pool, torch.uint8), _ptr(dst.vq_pool, torch.uint8),
                                  _ptr(dst.meta_pool, torch.int32), dst.n_pages_cap,
                                  _ptr(dst.page_table, torch.int32), dst.max_pages, _ptr(dst.remap, torch.int32),
                                  _ptr(dst.count, torch.int32), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_compact_quant", code)
    return dst


def kvp_compact_paged_workspace_bytes(batch, n_kv_heads, src_max_pages) -> int:
    return _lib.kvp_compact_paged_workspace_bytes(batch, n_kv_heads, src_max_pages)


def kvp_compact_paged(src: PagedKV, now, reserve, dst: PagedKV, *, status, workspace=None, stream=None):
    B, H, _ = src.page_table.shape
    need = kvp_compact_paged_workspace_bytes(B, H, src.max_pages)
    ws = _ws(need, src.k_pool.device, workspace)
    code = _lib.kvp_compact_paged(B, H, src.head_dim, _ptr(src.k_pool), _ptr(src.v_pool),
                                  _ptr(src.expire_pool, torch.int32), src.n_pages_cap,
                                  _ptr(src.page_table, torch.int32), src.max_pages, _ptr(src.remap, torch.int32),
                                  _ptr(src.count, torch.int32), now, reserve, _ptr(dst.k_pool), _ptr(dst.v_pool),
                                  _ptr(dst.expire_pool, torch.int32), dst.n_pages_cap,
                                  _ptr(dst.page_table, torch.int32), dst.max_pages, _ptr(dst.remap, torch.int32),
                                  _ptr(dst.count, torch.int32), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_compact_paged", code)
    return dst


# --------------------------------------------------------------------------- append

def kvp_append(cache: PagedKV, k_new, v_new, pos, *, mode, score=None, tau=None, flag_step=None,
               window=WINDOW, delay=0, status, stream=None):
    """Writes the token at position `pos` (k_new, v_new [B, H, d]) into every (b, h)'s next slot."""
    B, H, d = k_new.shape
    code = _lib.kvp_append(mode, B, H, d, pos, _ptr(k_new, torch.bfloat16, "k_new"),
                           _ptr(v_new, torch.bfloat16, "v_new"), _ptr(score, torch.float32, "score", True),
                           _ptr(tau, torch.float32, "tau", True), _ptr(flag_step, torch.int32, "flag_step", True),
                           window, delay, _ptr(cache.k_pool), _ptr(cache.v_pool),
                           _ptr(cache.expire_pool, torch.int32), cache.n_pages_cap,
                           _ptr(cache.page_table, torch.int32), cache.max_pages, _ptr(cache.remap, torch.int32),
                           _ptr(cache.count, torch.int32), _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_append", code)


def kvp_append_devpos(cache: PagedKV, k_new, v_new, pos_dev, *, mode, score=None, tau=None, flag_step=None,
                      window=WINDOW, delay=0, status, stream=None):
    """kvp_append with the position taken from pos_dev (a device int32 tensor of one element) when the call
    runs on the stream, so that one captured CUDA graph serves every decode step."""
    B, H, d = k_new.shape
    code = _lib.kvp_append_devpos(mode, B, H, d, _ptr(pos_dev, torch.int32, "pos_dev"),
                                  _ptr(k_new, torch.bfloat16, "k_new"),
                                  _ptr(v_new, torch.bfloat16, "v_new"), _ptr(score, torch.float32, "score", True),
                                  _ptr(tau, torch.float32, "tau", True),
                                  _ptr(flag_step, torch.int32, "flag_step", True),
                                  window, delay, _ptr(cache.k_pool), _ptr(cache.v_pool),
                                  _ptr(cache.expire_pool, torch.int32), cache.n_pages_cap,
                                  _ptr(cache.page_table, torch.int32), cache.max_pages,
                                  _ptr(cache.remap, torch.int32), _ptr(cache.count, torch.int32),
                                  _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_append_devpos", code)


def kvp_append_quant(qcache: QuantPagedKV, k_new, v_new, pos, *, score=None, tau=None, tau_q=None,
                     mode=KVP_MASK_KVZAP, flag_step=None, delay=0, window=WINDOW, status, stream=None):
    """Writes the token at position `pos` (k_new, v_new [B, H, d]) into the fp8 tier of every (b, h) whose
    score falls in [tau_q, tau) (or, mode KVP_MASK_DMS, whose flag_step [B, H] is >= 0)."""
    B, H, d = k_new.shape
    code = _lib.kvp_append_quant(mode, B, H, d, pos, _ptr(k_new, torch.bfloat16, "k_new"),
                                 _ptr(v_new, torch.bfloat16, "v_new"), _ptr(score, torch.float32, "score", True),
                                 _ptr(tau, torch.float32, "tau", True), _ptr(tau_q, torch.float32, "tau_q", True),
                                 _ptr(flag_step, torch.int32, "flag_step", True), window, delay,
                                 _ptr(qcache.kq_pool, torch.uint8),
                                 _ptr(qcache.vq_pool, torch.uint8), _ptr(qcache.meta_pool, torch.int32),
                                 qcache.n_pages_cap, _ptr(qcache.page_table, torch.int32), qcache.max_pages,
                                 _ptr(qcache.remap, torch.int32), _ptr(qcache.count, torch.int32),
                                 _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_append_quant", code)


# --------------------------------------------------------------------------- attention

def kvp_decode_attn_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim) -> int:
    return _lib.kvp_decode_attn_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim)


def kvp_decode_attn(q, cache: PagedKV, now, *, scale=0.0, out=None, grid_limit=0, workspace=None,
                    status=None, stream=None):
    """out[B, Hq, d] fp32 = attention of q [B, Hq, d] (bf16) over the slots of `cache` present at `now`.
    A caller-provided workspace must be zero-filled before its first use (torch.zeros); calls that record
    no error leave it that way."""
    B, Hq, d = q.shape
    H = cache.count.shape[1]
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    need = kvp_decode_attn_workspace_bytes(B, Hq, H, d)
    if workspace is None:
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=q.device)  # zero-filled before first use
    else:
        ws = _ws(need, q.device, workspace)
    code = _lib.kvp_decode_attn(B, Hq, H, d, _ptr(q, torch.bfloat16, "q"), _ptr(cache.k_pool),
                                _ptr(cache.v_pool), _ptr(cache.expire_pool, torch.int32), cache.n_pages_cap,
                                _ptr(cache.page_table, torch.int32), cache.max_pages,
                                _ptr(cache.count, torch.int32), now, float(scale), _ptr(out, torch.float32, "out"),
                                grid_limit, ws.data_ptr(), ws.numel() * ws.element_size(),
                                _ptr(status, torch.int32, "status", True), _stream(stream))
    _check("kvp_decode_attn", code)
    return out


def kvp_decode_attn_lse(q, cache: PagedKV, now, *, scale=0.0, out=None, lse=None, grid_limit=0, workspace=None,
                        status=None, stream=None):
    """(out, lse): kvp_decode_attn's out [B, Hq, d] fp32 and each row's log-sum-exp lse [B, Hq] fp32 (ln of the
    sum of exp(scale q.k) over the present slots; -inf for an empty row). Workspace rules: kvp_decode_attn's."""
    B, Hq, d = q.shape
    H = cache.count.shape[1]
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = kvp_decode_attn_workspace_bytes(B, Hq, H, d)
    if workspace is None:
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=q.device)  # zero-filled before first use
    else:
        ws = _ws(need, q.device, workspace)
    code = _lib.kvp_decode_attn_lse(B, Hq, H, d, _ptr(q, torch.bfloat16, "q"), _ptr(cache.k_pool),
                                    _ptr(cache.v_pool), _ptr(cache.expire_pool, torch.int32), cache.n_pages_cap,
                                    _ptr(cache.page_table, torch.int32), cache.max_pages,
                                    _ptr(cache.count, torch.int32), now, float(scale),
                                    _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"),
                                    grid_limit, ws.data_ptr(), ws.numel() * ws.element_size(),
                                    _ptr(status, torch.int32, "status", True), _stream(stream))
    _check("kvp_decode_attn_lse", code)
    return out, lse


def kvp_attn_merge(outs, lses, *, out=None, lse=None, stream=None):
    """(out, lse) of attention over the union of disjoint parts, from each part's rows: outs [P, ..., d] fp32 and
    lses [P, ...] fp32 (kvp_decode_attn_lse's, stacked). out [..., d], lse [...]."""
    n_parts, d = outs.shape[0], outs.shape[-1]
    if lses.shape != outs.shape[:-1]:
        raise ValueError("lses must have the shape of outs without its last dimension")
    rows = lses[0].numel()
    if out is None:
        out = torch.empty(outs.shape[1:], dtype=torch.float32, device=outs.device)
    if lse is None:
        lse = torch.empty(lses.shape[1:], dtype=torch.float32, device=outs.device)
    code = _lib.kvp_attn_merge(n_parts, rows, d, _ptr(outs, torch.float32, "outs"), _ptr(lses, torch.float32, "lses"),
                               _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"), _stream(stream))
    _check("kvp_attn_merge", code)
    return out, lse


def kvp_decode_attn_devpos(q, cache: PagedKV, now_dev, *, scale=0.0, out=None, grid_limit=0, workspace=None,
                           status=None, stream=None):
    """kvp_decode_attn with the decode position taken from now_dev (a device int32 tensor of one element)
    when the call runs on the stream. Workspace rules: kvp_decode_attn's."""
    B, Hq, d = q.shape
    H = cache.count.shape[1]
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    need = kvp_decode_attn_workspace_bytes(B, Hq, H, d)
    if workspace is None:
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=q.device)  # zero-filled before first use
    else:
        ws = _ws(need, q.device, workspace)
    code = _lib.kvp_decode_attn_devpos(B, Hq, H, d, _ptr(q, torch.bfloat16, "q"), _ptr(cache.k_pool),
                                       _ptr(cache.v_pool), _ptr(cache.expire_pool, torch.int32), cache.n_pages_cap,
                                       _ptr(cache.page_table, torch.int32), cache.max_pages,
                                       _ptr(cache.count, torch.int32), _ptr(now_dev, torch.int32, "now_dev"),
                                       float(scale), _ptr(out, torch.float32, "out"),
                                       grid_limit, ws.data_ptr(), ws.numel() * ws.element_size(),
                                       _ptr(status, torch.int32, "status", True), _stream(stream))
    _check("kvp_decode_attn_devpos", code)
    return out


def kvp_decode_attn_two_tier(q, cache: PagedKV, qcache: QuantPagedKV, now, *, scale=0.0, out=None, grid_limit=0,
                             workspace=None, status=None, stream=None):
    """Attention of q [B, Hq, d] over the bf16 tier `cache` (slots with now < expire) and the fp8 tier
    `qcache` (slots with now >= start, dequantized) -> out [B, Hq, d] fp32."""
    B, Hq, d = q.shape
    H = cache.count.shape[1]
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    need = kvp_decode_attn_workspace_bytes(B, Hq, H, d)
    if workspace is None:
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=q.device)  # zero-filled before first use
    else:
        ws = _ws(need, q.device, workspace)
    code = _lib.kvp_decode_attn_two_tier(
        B, Hq, H, d, _ptr(q, torch.bfloat16, "q"), _ptr(cache.k_pool), _ptr(cache.v_pool),
        _ptr(cache.expire_pool, torch.int32), cache.n_pages_cap, _ptr(cache.page_table, torch.int32),
        cache.max_pages, _ptr(cache.count, torch.int32), _ptr(qcache.kq_pool, torch.uint8),
        _ptr(qcache.vq_pool, torch.uint8), _ptr(qcache.meta_pool, torch.int32), qcache.n_pages_cap,
        _ptr(qcache.page_table, torch.int32), qcache.max_pages, _ptr(qcache.count, torch.int32), now, float(scale),
        _ptr(out, torch.float32, "out"), grid_limit, ws.data_ptr(), ws.numel() * ws.element_size(),
        _ptr(status, torch.int32, "status", True), _stream(stream))
    _check("kvp_decode_attn_two_tier", code)
    return out


def kvp_selftest_wait(limit_ns, *, status, waited_us=None, stream=None):
    """One warp waits on an mbarrier that nothing arrives on, with the bounded wait every kernel uses: after
    limit_ns it records KVP_ERR_TIMEOUT in status (device int32) and returns; waited_us (device uint32 [1], or
    None) receives how long the wait lasted."""
    code = _lib.kvp_selftest_wait(int(limit_ns), _ptr(status, torch.int32, "status"),
                                  _ptr(waited_us, None, "waited_us", True), _stream(stream))
    _check("kvp_selftest_wait", code)


# --------------------------------------------------------------------------- MLA latent cache

@dataclass
class LatentPagedKV:
    """Device buffers of one compacted MLA latent cache: one "kv head", one pool of latent rows."""
    pool: torch.Tensor          # bf16 [n_pages_cap, 16, 576]
    expire_pool: torch.Tensor   # int32 [n_pages_cap, 16]
    page_table: torch.Tensor    # int32 [B, max_pages]
    remap: torch.Tensor         # int32 [B, max_pages * 16]
    count: torch.Tensor         # int32 [B]

    @staticmethod
    def allocate(batch, n_pages_cap, max_pages, device="cuda"):
        return LatentPagedKV(
            torch.zeros((n_pages_cap, PAGE, LATENT_ROW), dtype=torch.bfloat16, device=device),
            torch.zeros((n_pages_cap, PAGE), dtype=torch.int32, device=device),
            torch.full((batch, max_pages), -1, dtype=torch.int32, device=device),
            torch.full((batch, max_pages * PAGE), -1, dtype=torch.int32, device=device),
            torch.zeros((batch,), dtype=torch.int32, device=device),
        )

    @property
    def n_pages_cap(self):
        return self.pool.shape[0]

    @property
    def max_pages(self):
        return self.page_table.shape[1]

    @property
    def batch(self):
        return self.count.shape[0]


def kvp_compact_latent(lat, now, reserve, dst: LatentPagedKV, *, mode, scores=None, tau=None, flag_step=None,
                       window=WINDOW, delay=0, status, workspace=None, stream=None):
    """Dense latent rows [B, T, 576] (row contiguous) with the mask applied on the fly: KVzap scores [B, T]
    (or [B*T, 1]) + tau [B], or DMS flag_step [B, T] -> dst."""
    B, T, R = lat.shape
    if lat.dtype != torch.bfloat16 or not lat.is_cuda or lat.stride(2) != 1:
        raise TypeError("lat must be a CUDA bf16 tensor with contiguous rows")
    if scores is not None and scores.numel() != B * T:
        raise ValueError("scores must hold B*T values")
    if flag_step is not None and flag_step.numel() != B * T:
        raise ValueError("flag_step must hold B*T values")
    if tau is not None and tau.numel() != B:
        raise ValueError("tau must hold B values")
    ws = _ws(kvp_compact_workspace_bytes(B, 1, T), lat.device, workspace)
    code = _lib.kvp_compact_latent(mode, B, R, T, lat.data_ptr(), lat.stride(0), lat.stride(1),
                                   _ptr(scores, torch.float32, "scores", True), _ptr(tau, torch.float32, "tau", True),
                                   _ptr(flag_step, torch.int32, "flag_step", True), window, delay, now, reserve,
                                   _ptr(dst.pool, torch.bfloat16), _ptr(dst.expire_pool, torch.int32),
                                   dst.n_pages_cap, _ptr(dst.page_table, torch.int32), dst.max_pages,
                                   _ptr(dst.remap, torch.int32), _ptr(dst.count, torch.int32), ws.data_ptr(),
                                   ws.numel() * ws.element_size(), _ptr(status, torch.int32, "status"),
                                   _stream(stream))
    _check("kvp_compact_latent", code)
    return dst


def kvp_compact_latent_paged(src: LatentPagedKV, now, reserve, dst: LatentPagedKV, *, status, workspace=None,
                             stream=None):
    """Re-compaction of a latent cache: its slots present at `now`, in slot order, into dst."""
    B = src.batch
    ws = _ws(kvp_compact_paged_workspace_bytes(B, 1, src.max_pages), src.pool.device, workspace)
    code = _lib.kvp_compact_latent_paged(B, src.pool.shape[2], _ptr(src.pool, torch.bfloat16),
                                         _ptr(src.expire_pool, torch.int32), src.n_pages_cap,
                                         _ptr(src.page_table, torch.int32), src.max_pages,
                                         _ptr(src.remap, torch.int32), _ptr(src.count, torch.int32), now, reserve,
                                         _ptr(dst.pool, torch.bfloat16), _ptr(dst.expire_pool, torch.int32),
                                         dst.n_pages_cap, _ptr(dst.page_table, torch.int32), dst.max_pages,
                                         _ptr(dst.remap, torch.int32), _ptr(dst.count, torch.int32), ws.data_ptr(),
                                         ws.numel() * ws.element_size(), _ptr(status, torch.int32, "status"),
                                         _stream(stream))
    _check("kvp_compact_latent_paged", code)
    return dst


def kvp_append_latent(cache: LatentPagedKV, lat_new, pos, *, mode, score=None, tau=None, flag_step=None,
                      window=WINDOW, delay=0, status, stream=None):
    """Writes the token at position `pos` (lat_new [B, 576]) into every batch element's next slot."""
    B, R = lat_new.shape
    code = _lib.kvp_append_latent(mode, B, R, pos, _ptr(lat_new, torch.bfloat16, "lat_new"),
                                  _ptr(score, torch.float32, "score", True), _ptr(tau, torch.float32, "tau", True),
                                  _ptr(flag_step, torch.int32, "flag_step", True), window, delay,
                                  _ptr(cache.pool, torch.bfloat16), _ptr(cache.expire_pool, torch.int32),
                                  cache.n_pages_cap, _ptr(cache.page_table, torch.int32), cache.max_pages,
                                  _ptr(cache.remap, torch.int32), _ptr(cache.count, torch.int32),
                                  _ptr(status, torch.int32, "status"), _stream(stream))
    _check("kvp_append_latent", code)


def kvp_decode_attn_mla_workspace_bytes(batch, n_q_heads, n_splits=0) -> int:
    return _lib.kvp_decode_attn_mla_workspace_bytes(batch, n_q_heads, n_splits)


def kvp_decode_attn_mla(q, cache: LatentPagedKV, now, *, scale=0.0, out=None, n_splits=0, workspace=None,
                        status=None, stream=None):
    """out[B, Hq, 512] fp32 = absorbed MLA attention of q [B, Hq, 576] (bf16) over the latent slots of `cache`
    present at `now`. The workspace needs no clearing between calls."""
    B, Hq, R = q.shape
    if R != LATENT_ROW:
        raise ValueError(f"q rows must hold {LATENT_ROW} values")
    if out is None:
        out = torch.empty((B, Hq, KVP_MLA_LATENT_DIM), dtype=torch.float32, device=q.device)
    need = kvp_decode_attn_mla_workspace_bytes(B, Hq, n_splits)
    ws = _ws(need, q.device, workspace)
    code = _lib.kvp_decode_attn_mla(B, Hq, KVP_MLA_LATENT_DIM, KVP_MLA_ROPE_DIM, _ptr(q, torch.bfloat16, "q"),
                                    _ptr(cache.pool, torch.bfloat16), _ptr(cache.expire_pool, torch.int32),
                                    cache.n_pages_cap, _ptr(cache.page_table, torch.int32), cache.max_pages,
                                    _ptr(cache.count, torch.int32), now, float(scale),
                                    _ptr(out, torch.float32, "out"), n_splits, ws.data_ptr(),
                                    ws.numel() * ws.element_size(), _ptr(status, torch.int32, "status", True),
                                    _stream(stream))
    _check("kvp_decode_attn_mla", code)
    return out


# --------------------------------------------------------------------------- block-scaled 8-bit cache
#
# These calls are made once a layer and step, often on little work, so their checks are written to be cheap: a device
# is its index, a handle checks its buffers when it is made and keeps their sizes (they cannot be replaced in it).

# (the names are looked up when called: torch builds without CUDA lack them, and the package imports there, too)
def _raw_stream(dev):
    """The current stream of a device, without a Stream object."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _current_device():
    return torch._C._cuda_getDevice()


def _refuse(t, dtype, name, dev, shape=None):
    """The error of a tensor that _on or _rows does not take."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, not on {t.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be of shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous (of q, k, v and their outputs: its last dimension)")


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _on(t, dtype, name, dev, shape=None):
    """Device pointer of a contiguous tensor that has to be on CUDA device `dev` (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _refuse(t, dtype, name, dev, shape)
    return t.data_ptr()


def _rows(t, name, dev, shape=None):
    """(device pointer, strides) of a bf16 tensor on `dev` whose last dimension is contiguous; the strides are its outer
    dimensions', 0 for those of length 1 (whose stride says nothing)."""
    own, st = t.shape, t.stride()
    if (t.dtype is not _BF16 or t.get_device() != dev or st[-1] != 1 and own[-1] != 1
            or shape is not None and own != shape):
        _refuse(t, _BF16, name, dev, shape)
    if 1 in own:
        return t.data_ptr(), tuple(0 if n == 1 else x for n, x in zip(own[:-1], st))
    return t.data_ptr(), st[:-1]


def _status(status, dev):
    """Device pointer of the status word (None: NULL)."""
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status must hold one value")
    return _on(status, _I32, "status", dev)


def _call(fn, dev, stream, *args):
    """One library call on device `dev`, whichever device is current, and on `stream` or dev's current stream."""
    if stream is None:
        raw = _raw_stream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{dev}")
        raw = stream.cuda_stream
    else:
        raw = int(stream)
    if _current_device() == dev:
        code = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, raw)
    if code != KVP_OK:
        raise KvpError(fn.__name__, code)


def _new(make, shape, dtype, dev, stream):
    """A new tensor that work on `stream` may use at once: memory of that stream's own, filled in its order."""
    device = torch.device("cuda", dev)
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _space(nbytes, workspace, dev, stream, make=torch.empty):
    """The caller's workspace, checked, or a new one, and its size in bytes."""
    if workspace is None:
        n = max(nbytes, 16)
        return _new(make, n, torch.uint8, dev, stream), n
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{dev}")
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError("workspace too small")
    return workspace, have


@dataclass(frozen=True)
class Block8PagedKV:
    """Device buffers of one cache held in 8 bits, a power-of-two scale for each page's K rows and one for its V rows
    (value = code * scale). fmt is KVP_BLOCK8_E4M3 or KVP_BLOCK8_INT8."""
    kq_pool: torch.Tensor       # uint8 [n_pages_cap, 16, d] codes of K rows
    vq_pool: torch.Tensor       # uint8 [n_pages_cap, 16, d] codes of V rows
    scale_pool: torch.Tensor    # fp32 [n_pages_cap, 2]: K scale, V scale
    expire_pool: torch.Tensor   # int32 [n_pages_cap, 16]
    page_table: torch.Tensor    # int32 [B, H, max_pages]
    remap: torch.Tensor         # int32 [B, H, max_pages * 16]
    count: torch.Tensor         # int32 [B, H]
    fmt: int = KVP_BLOCK8_E4M3

    def __post_init__(self):
        if self.fmt not in (KVP_BLOCK8_E4M3, KVP_BLOCK8_INT8):
            raise ValueError("fmt must be KVP_BLOCK8_E4M3 or KVP_BLOCK8_INT8")
        if not self.kq_pool.is_cuda:
            raise ValueError("kq_pool must be a CUDA tensor")
        dev = self.kq_pool.get_device()
        if self.kq_pool.dim() != 3 or self.kq_pool.shape[1] != PAGE:
            raise ValueError("kq_pool must be [n_pages_cap, 16, d]")
        if self.page_table.dim() != 3:
            raise ValueError("page_table must be [B, H, max_pages]")
        cap, (b, h, width) = self.kq_pool.shape[0], self.page_table.shape
        _on(self.kq_pool, torch.uint8, "kq_pool", dev)
        _on(self.vq_pool, torch.uint8, "vq_pool", dev, self.kq_pool.shape)
        _on(self.scale_pool, torch.float32, "scale_pool", dev, (cap, 2))
        _on(self.expire_pool, torch.int32, "expire_pool", dev, (cap, PAGE))
        _on(self.page_table, torch.int32, "page_table", dev)
        _on(self.remap, torch.int32, "remap", dev, (b, h, width * PAGE))
        _on(self.count, torch.int32, "count", dev, (b, h))
        object.__setattr__(self, "_dims", (dev, self.fmt, b, h, self.kq_pool.shape[2], cap, width))

    @staticmethod
    def allocate(batch, n_kv_heads, head_dim, n_pages_cap, max_pages, fmt=KVP_BLOCK8_E4M3, device="cuda"):
        return Block8PagedKV(
            torch.zeros((n_pages_cap, PAGE, head_dim), dtype=torch.uint8, device=device),
            torch.zeros((n_pages_cap, PAGE, head_dim), dtype=torch.uint8, device=device),
            torch.zeros((n_pages_cap, 2), dtype=torch.float32, device=device),
            torch.zeros((n_pages_cap, PAGE), dtype=torch.int32, device=device),
            torch.full((batch, n_kv_heads, max_pages), -1, dtype=torch.int32, device=device),
            torch.full((batch, n_kv_heads, max_pages * PAGE), -1, dtype=torch.int32, device=device),
            torch.zeros((batch, n_kv_heads), dtype=torch.int32, device=device), fmt)

    @property
    def n_pages_cap(self):
        return self.kq_pool.shape[0]

    @property
    def max_pages(self):
        return self.page_table.shape[2]

    @property
    def head_dim(self):
        return self.kq_pool.shape[2]


def kvp_compact_block8_workspace_bytes(batch, n_kv_heads, n_pos, n_pages_cap) -> int:
    return _lib.kvp_compact_block8_workspace_bytes(batch, n_kv_heads, n_pos, n_pages_cap)


def kvp_compact_block8(k, v, now, reserve, dst: Block8PagedKV, *, mode, scores=None, tau=None, flag_step=None,
                       window=WINDOW, delay=0, status, workspace=None, stream=None):
    """Dense K, V [B, T, H, d] (any strides with d contiguous) with the mask applied on the fly (KVzap scores [B, T, H]
    or [B*T, H] + tau [B, H], or DMS flag_step [B, H, T]) -> dst, quantised page by page. Counts, page table and remap
    list are kvp_compact_masked's."""
    dev, fmt, B, H, d, cap, width = dst._dims
    T = k.shape[1]
    (kp, st), (vp, v_st) = _rows(k, "k", dev, (B, T, H, d)), _rows(v, "v", dev, (B, T, H, d))
    if v_st != st:
        raise ValueError("k and v need the same strides")
    if scores is not None and scores.numel() != B * T * H:
        raise ValueError("scores must hold B*T*H values")
    if tau is not None and tau.numel() != B * H:
        raise ValueError("tau must hold B*H values")
    if flag_step is not None and flag_step.numel() != B * H * T:
        raise ValueError("flag_step must hold B*H*T values")
    ws, ws_bytes = _space(kvp_compact_block8_workspace_bytes(B, H, T, cap), workspace, dev, stream)
    _call(_lib.kvp_compact_block8, dev, stream, fmt, mode, B, H, d, T, kp, vp, *st,
          _on(scores, torch.float32, "scores", dev), _on(tau, torch.float32, "tau", dev),
          _on(flag_step, torch.int32, "flag_step", dev), window, delay, now, reserve, dst.kq_pool.data_ptr(),
          dst.vq_pool.data_ptr(), dst.scale_pool.data_ptr(), dst.expire_pool.data_ptr(), cap,
          dst.page_table.data_ptr(), width, dst.remap.data_ptr(), dst.count.data_ptr(), ws.data_ptr(), ws_bytes,
          _status(status, dev))
    return dst


def _per_head(t, dtype, name, dev, n):
    """Device pointer of a contiguous tensor of n values (None: NULL)."""
    if t is None:
        return None
    if t.numel() != n:
        raise ValueError(f"{name} must hold B*H values")
    return _on(t, dtype, name, dev)


def _append_block8(fn, cache, k_new, v_new, pos, mode, score, tau, flag_step, window, delay, status, stream):
    dev, fmt, B, H, d, cap, width = cache._dims
    kp, (k0, k1) = _rows(k_new, "k_new", dev, (B, H, d))
    vp, (v0, v1) = _rows(v_new, "v_new", dev, (B, H, d))
    _call(fn, dev, stream, fmt, mode, B, H, d, pos, kp, vp, k0, k1, v0, v1, _per_head(score, _F32, "score", dev, B * H),
          _per_head(tau, _F32, "tau", dev, B * H), _per_head(flag_step, _I32, "flag_step", dev, B * H), window, delay,
          cache.kq_pool.data_ptr(), cache.vq_pool.data_ptr(), cache.scale_pool.data_ptr(),
          cache.expire_pool.data_ptr(), cap, cache.page_table.data_ptr(), width, cache.remap.data_ptr(),
          cache.count.data_ptr(), _status(status, dev))


def kvp_append_block8(cache: Block8PagedKV, k_new, v_new, pos, *, mode, score=None, tau=None, flag_step=None,
                      window=WINDOW, delay=0, status, stream=None):
    """Quantises the token at position `pos` (k_new, v_new [B, H, d], any strides with d contiguous) into every
    (b, h)'s next slot; a page whose scale has to grow is rounded to the new one."""
    _append_block8(_lib.kvp_append_block8, cache, k_new, v_new, pos, mode, score, tau, flag_step, window, delay, status,
                   stream)


def kvp_append_block8_devpos(cache: Block8PagedKV, k_new, v_new, pos_dev, *, mode, score=None, tau=None,
                             flag_step=None, window=WINDOW, delay=0, status, stream=None):
    """kvp_append_block8 with the position taken from pos_dev (a device int32 tensor of one element) when the call
    runs on the stream."""
    pos = _on(pos_dev, torch.int32, "pos_dev", cache._dims[0])
    _append_block8(_lib.kvp_append_block8_devpos, cache, k_new, v_new, pos, mode, score, tau, flag_step, window, delay,
                   status, stream)


def kvp_read_block8(cache: Block8PagedKV, first_slot, n_slots, *, k_out=None, v_out=None, status=None, stream=None):
    """(k, v): slots first_slot .. first_slot + n_slots - 1 of every (b, h) as bf16 [B, n_slots, H, d] rows (k_out and
    v_out, if given, may have any strides with d contiguous, the same for both); zero rows past the counts. With
    status None, a page id out of range raises nothing: its rows come back as zeros."""
    dev, fmt, B, H, d, cap, width = cache._dims
    shape = (B, n_slots, H, d)
    if n_slots < 0:
        raise ValueError("n_slots must not be negative")
    if k_out is None:
        k_out = _new(torch.empty, shape, torch.bfloat16, dev, stream)
    if v_out is None:
        v_out = _new(torch.empty, shape, torch.bfloat16, dev, stream)
    (kp, st), (vp, v_st) = _rows(k_out, "k_out", dev, shape), _rows(v_out, "v_out", dev, shape)
    if v_st != st:
        raise ValueError("k_out and v_out need the same strides")
    if status is None:
        status = _new(torch.zeros, 1, torch.int32, dev, stream)
    _call(_lib.kvp_read_block8, dev, stream, fmt, B, H, d, cache.kq_pool.data_ptr(), cache.vq_pool.data_ptr(),
          cache.scale_pool.data_ptr(), cap, cache.page_table.data_ptr(), width, cache.count.data_ptr(), first_slot,
          n_slots, kp, vp, *st, _status(status, dev))
    return k_out, v_out


def kvp_decode_attn_block8_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim) -> int:
    return _lib.kvp_decode_attn_block8_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim)


def _attn_block8(fn, q, cache, now, scale, out, lse, grid_limit, workspace, status, stream):
    dev, fmt, B, H, d, cap, width = cache._dims
    shape = q.shape
    if len(shape) != 3 or shape[0] != B or shape[2] != d:
        raise ValueError("q must be [B, Hq, d] of the cache's batch and head_dim")
    Hq = shape[1]
    qp = _on(q, torch.bfloat16, "q", dev)
    if out is None:
        out = _new(torch.empty, shape, torch.float32, dev, stream)
    ws, ws_bytes = _space(_lib.kvp_decode_attn_block8_workspace_bytes(B, Hq, H, d), workspace, dev, stream, torch.zeros)
    _call(fn, dev, stream, fmt, B, Hq, H, d, qp, cache.kq_pool.data_ptr(), cache.vq_pool.data_ptr(),
          cache.scale_pool.data_ptr(), cache.expire_pool.data_ptr(), cap, cache.page_table.data_ptr(), width,
          cache.count.data_ptr(), now, scale, _on(out, torch.float32, "out", dev, shape),
          _on(lse, torch.float32, "lse", dev, (B, Hq)), grid_limit, ws.data_ptr(), ws_bytes, _status(status, dev))
    return out


def kvp_decode_attn_block8(q, cache: Block8PagedKV, now, *, scale=0.0, out=None, lse=None, grid_limit=0,
                           workspace=None, status=None, stream=None):
    """out[B, Hq, d] fp32 = attention of q [B, Hq, d] (bf16) over the slots of the 8-bit `cache` present at `now`; lse
    (fp32 [B, Hq], if given) receives each row's log-sum-exp, for kvp_attn_merge. A caller-provided workspace must be
    zero-filled before its first use (torch.zeros); every call leaves it ready for the next one, of whatever sizes."""
    return _attn_block8(_lib.kvp_decode_attn_block8, q, cache, now, scale, out, lse, grid_limit, workspace, status,
                        stream)


def kvp_decode_attn_block8_devpos(q, cache: Block8PagedKV, now_dev, *, scale=0.0, out=None, lse=None, grid_limit=0,
                                  workspace=None, status=None, stream=None):
    """kvp_decode_attn_block8 with the decode position taken from now_dev (a device int32 tensor of one element) when
    the call runs on the stream."""
    now = _on(now_dev, torch.int32, "now_dev", cache._dims[0])
    return _attn_block8(_lib.kvp_decode_attn_block8_devpos, q, cache, now, scale, out, lse, grid_limit, workspace,
                        status, stream)


# --------------------------------------------------------------------------- norm and rotation of queries and keys

def kvp_rope_turns(inv_freq, *, device=None):
    """inv_freq (radians per position, a sequence or tensor of magnitudes up to 2^32; taken as float64) as the table that
    kvp_qk_norm_rope takes: 64-bit fractions of a turn, an int64 tensor on `device` (inv_freq's, if it is on a GPU)."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64)
    if device is None:
        device = f.device if f.is_cuda else torch.device("cuda")
    f = f.detach().cpu().contiguous()
    turns = torch.empty(f.numel(), dtype=torch.int64)
    _check("kvp_rope_turns", _lib.kvp_rope_turns(f.numel(), f.data_ptr(), turns.data_ptr()))
    return turns.to(device)


def _head_rows(x, y, name, dev, n, d, stream):
    """(heads, in, its strides, out, its strides) of q or k for kvp_qk_norm_rope, and the output."""
    if x is None:
        if y is not None:
            raise ValueError(f"{name}_out without {name}")
        return 0, None, (0, 0), None, (0, 0), None
    shape = x.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != d:
        raise ValueError(f"{name} must be [n, heads, d]")
    if y is None:
        y = _new(torch.empty, shape, _BF16, dev, stream)
    xp, xs = _rows(x, name, dev)
    yp, ys = _rows(y, name + "_out", dev, shape)
    return shape[1], xp, xs, yp, ys, y


def kvp_qk_norm_rope(q, k, pos, turns, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                     k_out=None, stream=None):
    """(q_out, k_out): the heads of q [n, Hq, d] and k [n, Hk, d] (bf16, any strides with d contiguous; either may be
    None), each row normed (weights fp32 [d], None: no norm) and its first 2 * len(turns) values rotated by its token's
    position (pos int32 [n]; turns from kvp_rope_turns, None: no rotation; interleaved: pairs (2i, 2i + 1) instead of
    (i, i + len(turns))). q_out and k_out may be q and k themselves."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is required")
    dev, shape = some.get_device(), some.shape
    if dev < 0:
        raise ValueError("q and k must be CUDA tensors")
    n, d = shape[0], shape[-1]
    rot = 0
    if turns is not None:
        rot = 2 * turns.numel()
        if pos is None:
            raise ValueError("pos is required with turns")
    hq, qp, (q0, q1), qo, (qo0, qo1), q_out = _head_rows(q, q_out, "q", dev, n, d, stream)
    hk, kp, (k0, k1), ko, (ko0, ko1), k_out = _head_rows(k, k_out, "k", dev, n, d, stream)
    _call(_lib.kvp_qk_norm_rope, dev, stream, n, hq, hk, d, rot, interleaved, qp, q0, q1, kp, k0, k1,
          _on(pos, _I32, "pos", dev, (n,)) if rot else None, _on(turns, torch.int64, "turns", dev) if rot else None,
          _on(q_weight, _F32, "q_weight", dev, (d,)), _on(k_weight, _F32, "k_weight", dev, (d,)), eps, qo, qo0, qo1, ko,
          ko0, ko1)
    return q_out, k_out


# --------------------------------------------------------------------------- attention over prompts, eviction by its weights
#
# Tensors are checked as in the two sections above: on one CUDA device, which need not be the current one.

def _device_of(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _seqs(seq_start, seq_len, dev):
    """(number of sequences, pointer of the starts, pointer of the lengths or None)."""
    n = seq_start.numel() - 1
    if n < 0 or seq_start.dim() != 1:
        raise ValueError("seq_start must be [n_seqs + 1]")
    return n, _on(seq_start, _I32, "seq_start", dev), _on(seq_len, _I32, "seq_len", dev, (n,))


def kvp_prompt_attn(q, k, v, seq_start, *, seq_len=None, scale=0.0, out=None, lse=None, status=None, stream=None):
    """out [n_tok, Hq, d] bf16 = causal attention of q [n_tok, Hq, d] over k, v [n_tok, H, d] (bf16, any strides with d
    contiguous: views of one projection need no copy), each packed sequence over itself: rows seq_start[s] ..
    seq_start[s + 1] - 1 (int32 [n_seqs + 1]), or the first seq_len[s] of them (int32 [n_seqs]). lse (fp32 [Hq, n_tok],
    if given) receives each row's log-sum-exp, for kvp_prompt_weights."""
    dev = _device_of(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [n_tok, heads, d]")
    (n, hq, d), h = q.shape, k.shape[1]
    qp, qs = _rows(q, "q", dev)
    kp, ks = _rows(k, "k", dev, (n, h, d))
    vp, vs = _rows(v, "v", dev, (n, h, d))
    if out is None:
        out = _new(torch.empty, (n, hq, d), _BF16, dev, stream)
    op, os_ = _rows(out, "out", dev, (n, hq, d))
    n_seqs, sp, lp = _seqs(seq_start, seq_len, dev)
    _call(_lib.kvp_prompt_attn, dev, stream, n_seqs, n, hq, h, d, qp, *qs, kp, *ks, vp, *vs, sp, lp, scale, op, *os_,
          _on(lse, _F32, "lse", dev, (hq, n)), _status(status, dev))
    return out


def kvp_prompt_weights(q, k, seq_start, lse, *, seq_len=None, scale=0.0, n_last=0, acc=None, status=None, stream=None):
    """acc fp32: the weight that each key of k [n_tok, H, d] received from the queries q [n_tok, Hq, d] of its sequence
    (the last n_last of each sequence, 0: all), given kvp_prompt_attn's lse [Hq, n_tok]; a query whose lse is -inf pays
    nothing, whatever it holds. acc is [n_tok, H] (the scores that kvp_threshold and kvp_compact_masked take, where sequences
    are of one length) or [n_seqs, H, T] (the sums by position that kvp_evict and kvp_decode_attn_acc take, T at least the
    longest sequence), of any strides; None: a new [n_tok, H], zero in rows of no sequence."""
    dev = _device_of(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [n_tok, heads, d]")
    (n, hq, d), h = q.shape, k.shape[1]
    qp, qs = _rows(q, "q", dev)
    kp, ks = _rows(k, "k", dev, (n, h, d))
    n_seqs, sp, lp = _seqs(seq_start, seq_len, dev)
    if acc is None:
        acc = _new(torch.zeros, (n, h), _F32, dev, stream)
    by_token = acc.dim() == 2
    if acc.shape != (n, h) if by_token else acc.dim() != 3 or acc.shape[:2] != (n_seqs, h):
        raise ValueError("acc must be [n_tok, H] or [n_seqs, H, T]")
    if acc.dtype is not _F32 or acc.get_device() != dev:
        _refuse(acc, _F32, "acc", dev)
    st = acc.stride()
    strides = (-1, st[0], st[1], 0) if by_token else (st[0], st[2], st[1], acc.shape[2])
    _call(_lib.kvp_prompt_weights, dev, stream, n_seqs, n, hq, h, d, qp, *qs, kp, *ks, sp, lp,
          _on(lse, _F32, "lse", dev, (hq, n)), scale, n_last, acc.data_ptr(), *strides, _status(status, dev))
    return acc


def _sums(acc, dev, b, h):
    """(pointer, stride of b, stride of h, length) of weight sums [B, H, T] whose positions lie side by side."""
    if acc.dim() != 3 or acc.shape[:2] != (b, h):
        raise ValueError("acc must be [B, H, T]")
    st, t = acc.stride(), acc.shape[2]
    if acc.dtype is not _F32 or acc.get_device() != dev or (st[2] != 1 and t > 1):
        _refuse(acc, _F32, "acc", dev)
    return acc.data_ptr(), st[0] if b > 1 else 0, st[1] if h > 1 else 0, t


def kvp_decode_attn_acc_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim, max_pages) -> int:
    return _lib.kvp_decode_attn_acc_workspace_bytes(batch, n_q_heads, n_kv_heads, head_dim, max_pages)


def _attn_acc(fn, q, cache, now, acc, scale, out, lse, grid_limit, workspace, status, stream):
    dev, shape = _device_of(q, "q"), q.shape
    cap, d = cache.k_pool.shape[0], cache.k_pool.shape[-1]
    b, h, width = cache.page_table.shape
    if len(shape) != 3 or shape[0] != b or shape[2] != d:
        raise ValueError("q must be [B, Hq, d] of the cache's batch and head_dim")
    hq, pool = shape[1], (cap, PAGE, d)
    if out is None:
        out = _new(torch.empty, shape, _F32, dev, stream)
    ws, ws_bytes = _space(_lib.kvp_decode_attn_acc_workspace_bytes(b, hq, h, d, width), workspace, dev, stream,
                          torch.zeros)
    _call(fn, dev, stream, b, hq, h, d, _on(q, _BF16, "q", dev), _on(cache.k_pool, _BF16, "k_pool", dev, pool),
          _on(cache.v_pool, _BF16, "v_pool", dev, pool), _on(cache.expire_pool, _I32, "expire_pool", dev, (cap, PAGE)),
          cap, _on(cache.page_table, _I32, "page_table", dev), width,
          _on(cache.remap, _I32, "remap", dev, (b, h, width * PAGE)), _on(cache.count, _I32, "count", dev, (b, h)), now,
          scale, _on(out, _F32, "out", dev, shape), _on(lse, _F32, "lse", dev, (b, hq)), *_sums(acc, dev, b, h),
          grid_limit, ws.data_ptr(), ws_bytes, _status(status, dev))
    return out


def kvp_decode_attn_acc(q, cache: PagedKV, now, acc, *, scale=0.0, out=None, lse=None, grid_limit=0, workspace=None,
                        status=None, stream=None):
    """kvp_decode_attn_lse (lse optional) that adds the weights it pays, over the query heads of a kv head, to
    acc[b, h, position] (fp32 [B, H, T], positions side by side; zeros where none has been paid yet). A caller-provided
    workspace must be zero-filled before its first use (torch.zeros), and again after a call that recorded an error; after a
    time-out the sums are as they were before the call."""
    return _attn_acc(_lib.kvp_decode_attn_acc, q, cache, now, acc, scale, out, lse, grid_limit, workspace, status, stream)


def kvp_decode_attn_acc_devpos(q, cache: PagedKV, now_dev, acc, *, scale=0.0, out=None, lse=None, grid_limit=0,
                               workspace=None, status=None, stream=None):
    """kvp_decode_attn_acc with the decode position taken from now_dev (a device int32 tensor of one element) when the
    call runs on the stream."""
    now = _on(now_dev, _I32, "now_dev", _device_of(q, "q"))
    return _attn_acc(_lib.kvp_decode_attn_acc_devpos, q, cache, now, acc, scale, out, lse, grid_limit, workspace, status,
                     stream)


def kvp_evict(acc, now, *, budget, recent=WINDOW, expire=None, count=None, stream=None):
    """(expire int32 [B, H, T], count int32 [B, H]) from weight sums acc (fp32 [B, H, T], any strides): of each (b, h)
    the last `recent` positions stay, and of the others the heaviest that `budget` leaves room for (the first of equal
    ones). expire is EXPIRE_NEVER for those and `now` for the rest: kvp_compact at step `now` drops them."""
    dev = _device_of(acc, "acc")
    if acc.dim() != 3:
        raise ValueError("acc must be [B, H, T]")
    if acc.dtype is not _F32:
        _refuse(acc, _F32, "acc", dev)
    b, h, t = acc.shape
    if expire is None:
        expire = _new(torch.empty, (b, h, t), _I32, dev, stream)
    if count is None:
        count = _new(torch.empty, (b, h), _I32, dev, stream)
    st = acc.stride()
    _call(_lib.kvp_evict, dev, stream, b, h, t, acc.data_ptr(), st[0], st[2], st[1], budget, recent, now,
          _on(expire, _I32, "expire", dev, (b, h, t)), _on(count, _I32, "count", dev, (b, h)))
    return expire, count


def _evict_paged(fn, cache, acc, now, dev, budget, recent, kept, status, stream):
    table = cache.page_table
    b, h, width = table.shape if table.dim() == 3 else (table.shape[0], 1, table.shape[1])   # (a latent cache has no heads)
    cap = cache.expire_pool.shape[0]
    heads = table.shape[:-1]
    _call(fn, dev, stream, b, h, *_sums(acc, dev, b, h), _on(cache.expire_pool, _I32, "expire_pool", dev, (cap, PAGE)), cap,
          _on(table, _I32, "page_table", dev), width, _on(cache.remap, _I32, "remap", dev, (*heads, width * PAGE)),
          _on(cache.count, _I32, "count", dev, heads), budget, recent, now, _per_head(kept, _I32, "kept", dev, b * h),
          _status(status, dev))
    return cache


def kvp_evict_paged(cache, acc, now, *, budget, recent=WINDOW, kept=None, status=None, stream=None):
    """Entries of a paged cache in use (PagedKV, Block8PagedKV or LatentPagedKV) beyond the budget: of each (b, h)'s
    present slots those of the last `recent` positions stay, and of the others the heaviest by acc[b, h, position]
    (fp32 [B, H, T], positions side by side) that `budget` leaves room for; the rest expire at `now`. kept (int32
    [B, H], if given) receives how many stay."""
    return _evict_paged(_lib.kvp_evict_paged, cache, acc, now, _device_of(acc, "acc"), budget, recent, kept, status, stream)


def kvp_evict_paged_devpos(cache, acc, now_dev, *, budget, recent=WINDOW, kept=None, status=None, stream=None):
    """kvp_evict_paged with the step taken from now_dev (a device int32 tensor of one element) when the call runs on the
    stream."""
    dev = _device_of(acc, "acc")
    return _evict_paged(_lib.kvp_evict_paged_devpos, cache, acc, _on(now_dev, _I32, "now_dev", dev), dev, budget, recent,
                        kept, status, stream)


__all__ = [n for n in dir() if n.startswith(("kvp_", "KVP_", "PagedKV", "QuantPagedKV", "LatentPagedKV",
                                             "Block8PagedKV", "KvpError"))] + [
    "status_string", "version", "library", "PAGE", "WINDOW", "EXPIRE_NEVER", "LATENT_ROW"]
