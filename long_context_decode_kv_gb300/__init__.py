"""GB300-native Quest-style sparse decode attention over a long KV cache.

Thin Python binding over ``libkvdecode.so`` (C ABI in ``include/kvdecode.h``).
Every call marshals torch tensors to raw pointers and calls the library on the
tensor's CUDA stream; all arithmetic runs in the library's CUDA kernels.
PyTorch only provides device memory, streams and events.  There is no CPU
fallback: if the library is not built, loading it raises.

Entry points (same names as the C ABI, without the ``kvd_`` prefix):
  kv_append, select_blocks, decode_attn, decode_attn_dense, decode_step,
  decode_step_host, workspace_bytes, selected_count, status_string,
  debug_qk_int8, debug_scores, decode_attn_static; and around the decode
  rope_table (kvd_rope_freqs), qk_norm_rope, paged_append, paged_attn; over
  latent rows latent_append, latent_attn; and paged_mass, paged_evict (of
  either cache).
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

import torch

from . import synth  # noqa: F401  (seeded inputs; no method arithmetic)

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkvdecode.so")

F16 = 0
INT8 = 1
Q8_0 = 2
Q4_0 = 3
BF16 = 4  # paged caches only
BLOCK = 64
HEAD_DIM = 128

STATUS = {0: "KVD_OK", 1: "KVD_ERR_INVALID", 2: "KVD_ERR_UNSUPPORTED", 3: "KVD_ERR_CAPACITY",
          4: "KVD_ERR_CUDA", 5: "KVD_ERR_TIMEOUT", 6: "KVD_ERR_WORKSPACE"}

EXPORTS = ("kvd_kv_append", "kvd_select_blocks", "kvd_decode_attn", "kvd_decode_attn_dense",
           "kvd_decode_step", "kvd_decode_step_host", "kvd_workspace_bytes",
           "kvd_selected_count", "kvd_status_string", "kvd_abi_version", "kvd_debug_qk_int8",
           "kvd_debug_scores", "kvd_decode_attn_static", "kvd_decode_attn_sv",
           "kvd_decode_attn_tail", "kvd_kv_append_f32", "kvd_select_blocks_per_head",
           "kvd_decode_attn_per_head", "kvd_debug_wait_timeout", "kvd_debug_stage_marks",
           "kvd_rope_freqs", "kvd_qk_norm_rope", "kvd_paged_append", "kvd_paged_attn",
           "kvd_paged_workspace_bytes", "kvd_paged_attn_lse", "kvd_latent_append",
           "kvd_latent_attn", "kvd_latent_workspace_bytes", "kvd_paged_mass", "kvd_latent_mass",
           "kvd_paged_evict", "kvd_latent_evict")


class KvdError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} -> {STATUS.get(code, code)}")


class CacheStruct(C.Structure):
    """Mirror of ``kvd_cache``."""
    _fields_ = [("dtype", C.c_int32), ("batch", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("max_seq", C.c_int32), ("block", C.c_int32),
                ("len", C.c_int32), ("reserved", C.c_int32),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("kbounds", C.c_void_p), ("dev_status", C.c_void_p),
                ("moments", C.c_void_p), ("seq_lens", C.c_void_p)]


class PagedCacheStruct(C.Structure):
    """Mirror of ``kvd_paged_cache``."""
    _fields_ = [("dtype", C.c_int32), ("batch", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("n_pages", C.c_int32), ("page_size", C.c_int32),
                ("max_pages", C.c_int32), ("len", C.c_int32),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("page_table", C.c_void_p), ("seq_lens", C.c_void_p),
                ("dev_status", C.c_void_p)]


class LatentCacheStruct(C.Structure):
    """Mirror of ``kvd_latent_cache``."""
    _fields_ = [("dtype", C.c_int32), ("batch", C.c_int32), ("rank", C.c_int32),
                ("rope_dim", C.c_int32), ("n_pages", C.c_int32), ("page_size", C.c_int32),
                ("max_pages", C.c_int32), ("len", C.c_int32), ("rows", C.c_void_p),
                ("page_table", C.c_void_p), ("seq_lens", C.c_void_p), ("dev_status", C.c_void_p)]


class PartsStruct(C.Structure):
    """Mirror of ``kvd_head_parts``."""
    _fields_ = [("x", C.c_void_p), ("stride", C.c_int64), ("head_stride", C.c_int64),
                ("dtype", C.c_int32), ("n_heads", C.c_int32)]


class HeadsStruct(C.Structure):
    """Mirror of ``kvd_heads``."""
    _fields_ = [("x", C.c_void_p), ("stride", C.c_int64), ("dtype", C.c_int32),
                ("n_heads", C.c_int32)]


class RopeStruct(C.Structure):
    """Mirror of ``kvd_rope``."""
    _fields_ = [("freqs", C.c_void_p), ("rot_dim", C.c_int32), ("interleaved", C.c_int32),
                ("mscale", C.c_float), ("reserved", C.c_int32)]


_lib = None


def lib():
    """Load libkvdecode.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "long_context_decode_kv_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        p, i32, sz = C.c_void_p, C.c_int32, C.c_size_t
        cp = C.POINTER(CacheStruct)
        L.kvd_kv_append.argtypes = [cp, p, p, i32, p]
        L.kvd_kv_append_f32.argtypes = [cp, p, p, i32, p]
        L.kvd_select_blocks.argtypes = [cp, p, i32, i32, i32, i32, p, p, p, sz, p]
        L.kvd_decode_attn.argtypes = [cp, p, i32, C.c_float, p, p, i32, p, p, sz, p]
        L.kvd_decode_attn_dense.argtypes = [cp, p, i32, C.c_float, p, p, sz, p]
        L.kvd_decode_attn_static.argtypes = [cp, p, i32, C.c_float, p, p, i32, p, p]
        L.kvd_decode_attn_sv.argtypes = [cp, p, i32, C.c_float, p, p, i32, C.c_float, p, p, sz,
                                         p]
        L.kvd_select_blocks_per_head.argtypes = [cp, p, i32, i32, i32, i32, p, p, p, sz, p]
        L.kvd_decode_attn_per_head.argtypes = [cp, p, i32, C.c_float, p, p, i32, p, p, sz, p]
        L.kvd_decode_attn_tail.argtypes = [cp, p, i32, C.c_float, p, p, i32, p, p, sz, p]
        L.kvd_decode_step.argtypes = [cp, p, p, p, i32, C.c_float, i32, i32, i32, p, p, p, p,
                                      sz, p]
        L.kvd_decode_step_host.argtypes = [cp, p, p, p, i32, C.c_float, i32, i32, i32, p, p, p,
                                           p, sz, p]
        L.kvd_workspace_bytes.argtypes = [cp, i32]
        L.kvd_workspace_bytes.restype = sz
        L.kvd_selected_count.argtypes = [i32, i32, i32, i32, i32]
        L.kvd_selected_count.restype = i32
        L.kvd_status_string.argtypes = [i32]
        L.kvd_status_string.restype = C.c_char_p
        L.kvd_abi_version.restype = i32
        L.kvd_debug_qk_int8.argtypes = [cp, p, i32, p, p, p, p]
        L.kvd_debug_scores.argtypes = [cp, p, i32, p, p]
        L.kvd_debug_wait_timeout.argtypes = [p, i32, p]
        L.kvd_debug_stage_marks.argtypes = [p, sz]
        pc, hp, rp, f64 = C.POINTER(PagedCacheStruct), C.POINTER(HeadsStruct), \
            C.POINTER(RopeStruct), C.c_double
        L.kvd_rope_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, p, C.POINTER(C.c_float)]
        L.kvd_qk_norm_rope.argtypes = [hp, hp, hp, hp, i32, i32, p, rp, p, p, C.c_float, p]
        L.kvd_paged_append.argtypes = [pc, hp, hp, i32, p, rp, p, hp, hp, p, C.c_float, p]
        L.kvd_paged_attn.argtypes = [pc, hp, i32, p, i32, C.c_float, i32, hp, p, sz, p]
        L.kvd_paged_workspace_bytes.argtypes = [pc, i32, i32, i32]
        L.kvd_paged_workspace_bytes.restype = sz
        lc, qp, f32, i64 = C.POINTER(LatentCacheStruct), C.POINTER(PartsStruct), C.c_float, \
            C.c_int64
        L.kvd_paged_attn_lse.argtypes = [pc, hp, i32, p, i32, f32, i32, hp, p, p, sz, p]
        L.kvd_latent_append.argtypes = [lc, hp, hp, i32, p, rp, p, qp, qp, f32, p]
        L.kvd_latent_attn.argtypes = [lc, hp, i32, p, i32, f32, i32, hp, p, p, sz, p]
        L.kvd_latent_workspace_bytes.argtypes = [lc, i32, i32, i32]
        L.kvd_latent_workspace_bytes.restype = sz
        mass = [hp, p, i32, p, i32, f32, i32, p, i64, f32, p, i64, p]
        L.kvd_paged_mass.argtypes = [pc] + mass
        L.kvd_latent_mass.argtypes = [lc] + mass
        evict = [p, i64, i32, i32, i32, p, i32, p, p, p, i64, p]
        L.kvd_paged_evict.argtypes = [pc] + evict
        L.kvd_latent_evict.argtypes = [lc] + evict
        _lib = L
    return _lib


def _check(fn: str, rc: int):
    if rc != 0:
        raise KvdError(fn, rc)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor, stream=None):
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return C.c_void_p(stream.cuda_stream)


class KVCache:
    """Caller-owned cache tensors plus the C descriptor that points at them.

    k, v      [B, Hkv, max_seq, D]    float16 or int8 codes, or
              [B, Hkv, max_seq, D/2]  uint8 pairs of 4-bit codes (q4_0); D = head_dim:
              128, or any multiple of 16 up to 1024 for f16 / int8 caches without
              moments or seq_lens
    k_scale   [B, Hkv, max_seq]       float32 (int8), or
              [B, Hkv, max_seq, 4]    float16 group scales (q8_0, q4_0); same for v_scale
    kbounds   [B, Hkv, max_seq // 64, D, 2] float16: (kmin, kmax) per channel
    status    [1] int32 device word for device-side faults
    moments   [B, Hkv, max_seq // 64, 2, 128] float16 block means of K then V
              (only with moments=True: the moment tail of decode_attn_tail)
    seq_lens  optional [B] int32 device tensor of per-sequence lengths (each at
              most len; len is then the batch's maximum); see set_seq_lens
    """

    def __init__(self, dtype: int, batch: int, n_kv_heads: int, max_seq: int,
                 head_dim: int = HEAD_DIM, block: int = BLOCK, device="cuda",
                 tensors: Optional[dict] = None, moments: bool = False):
        self.dtype, self.batch, self.n_kv_heads = dtype, batch, n_kv_heads
        self.head_dim, self.max_seq, self.block = head_dim, max_seq, block
        dev = torch.device(device)
        if tensors is not None:
            self.t = dict(tensors)
        else:
            kvt = (torch.float16 if dtype == F16 else
                   torch.uint8 if dtype == Q4_0 else torch.int8)
            width = head_dim // 2 if dtype == Q4_0 else head_dim  # q4_0: two codes a byte
            nb = max_seq // block if block > 0 else 0
            self.t = {
                "k": torch.empty(batch, n_kv_heads, max_seq, width, dtype=kvt, device=dev),
                "v": torch.empty(batch, n_kv_heads, max_seq, width, dtype=kvt, device=dev),
                "kbounds": torch.empty(batch, n_kv_heads, nb, head_dim, 2, dtype=torch.float16,
                                       device=dev),
                "status": torch.zeros(1, dtype=torch.int32, device=dev),
            }
            if dtype == INT8:
                self.t["k_scale"] = torch.empty(batch, n_kv_heads, max_seq, dtype=torch.float32,
                                                device=dev)
                self.t["v_scale"] = torch.empty(batch, n_kv_heads, max_seq, dtype=torch.float32,
                                                device=dev)
            elif dtype in (Q8_0, Q4_0):
                ng = head_dim // 32
                self.t["k_scale"] = torch.empty(batch, n_kv_heads, max_seq, ng,
                                                dtype=torch.float16, device=dev)
                self.t["v_scale"] = torch.empty(batch, n_kv_heads, max_seq, ng,
                                                dtype=torch.float16, device=dev)
            if moments:
                self.t["moments"] = torch.empty(batch, n_kv_heads, nb, 2, head_dim,
                                                dtype=torch.float16, device=dev)
        self.s = CacheStruct(dtype, batch, n_kv_heads, head_dim, max_seq, block, 0, 0,
                             _ptr(self.t["k"]), _ptr(self.t["v"]),
                             _ptr(self.t.get("k_scale")), _ptr(self.t.get("v_scale")),
                             _ptr(self.t["kbounds"]), _ptr(self.t.get("status")),
                             _ptr(self.t.get("moments")))

    def set_seq_lens(self, seq_lens: Optional[torch.Tensor]):
        """Give every sequence its own length (an int32 [B] device tensor the
        caller owns and advances after each append), or None for one length."""
        if seq_lens is not None:
            assert seq_lens.dtype == torch.int32 and seq_lens.shape == (self.batch,)
            self.t["seq_lens"] = seq_lens
        else:
            self.t.pop("seq_lens", None)
        self.s.seq_lens = _ptr(seq_lens)

    def view(self, b: int) -> "KVCache":
        """Sequence b alone, as a batch-1 cache over the same memory (one
        sequence's rows, scales, bounds and means are contiguous slices)."""
        t = {k: v[b:b + 1] for k, v in self.t.items() if k not in ("status", "seq_lens")}
        t["status"] = self.t["status"]
        c = KVCache(self.dtype, 1, self.n_kv_heads, self.max_seq, self.head_dim, self.block,
                    device=self.t["k"].device, tensors=t)
        return c

    @property
    def kmin(self) -> torch.Tensor:
        """View [B, Hkv, max_seq // 64, 128] of the per-block channel minima."""
        return self.t["kbounds"][..., 0]

    @property
    def kmax(self) -> torch.Tensor:
        """View [B, Hkv, max_seq // 64, 128] of the per-block channel maxima."""
        return self.t["kbounds"][..., 1]

    @property
    def len(self) -> int:
        return self.s.len

    @len.setter
    def len(self, n: int):
        self.s.len = int(n)

    def __getattr__(self, name):
        t = self.__dict__.get("t")
        if t is not None and name in t:
            return t[name]
        raise AttributeError(name)

    def ref(self):
        return C.byref(self.s)

    def device_status(self) -> int:
        return int(self.t["status"].item())


def workspace_bytes(cache: KVCache, n_heads: int) -> int:
    return int(lib().kvd_workspace_bytes(cache.ref(), n_heads))


def make_workspace(cache: KVCache, n_heads: int) -> torch.Tensor:
    """A zero-filled, 256-byte aligned workspace for every call on this cache."""
    n = workspace_bytes(cache, n_heads)
    if n == 0:
        raise KvdError("kvd_workspace_bytes", 1)
    return torch.zeros(n, dtype=torch.uint8, device=cache.k.device)


def selected_count(length: int, k_sel: int, sink_tokens: int, recent_tokens: int,
                   block: int = BLOCK) -> int:
    return int(lib().kvd_selected_count(length, block, k_sel, sink_tokens, recent_tokens))


def status_string(code: int) -> str:
    return lib().kvd_status_string(code).decode()


def kv_append(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
    """k_new, v_new: [B, n_new, Hkv, D] float16 on the cache's device."""
    _check("kvd_kv_append", lib().kvd_kv_append(cache.ref(), _ptr(k_new), _ptr(v_new),
                                                int(k_new.shape[1]), _stream(k_new, stream)))


def kv_append_f32(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
    """k_new, v_new: [B, n_new, Hkv, D] float32 on the cache's device."""
    _check("kvd_kv_append_f32", lib().kvd_kv_append_f32(cache.ref(), _ptr(k_new), _ptr(v_new),
                                                        int(k_new.shape[1]),
                                                        _stream(k_new, stream)))


def select_blocks(cache: KVCache, q: torch.Tensor, k_sel: int, sink_tokens: int,
                  recent_tokens: int, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                  workspace: torch.Tensor, stream=None):
    _check("kvd_select_blocks", lib().kvd_select_blocks(
        cache.ref(), _ptr(q), int(q.shape[1]), k_sel, sink_tokens, recent_tokens,
        _ptr(sel_idx), _ptr(sel_cnt), _ptr(workspace), workspace.numel(), _stream(q, stream)))


def decode_attn(cache: KVCache, q: torch.Tensor, softmax_scale: float, sel_idx: torch.Tensor,
                sel_cnt: torch.Tensor, max_sel: int, out: torch.Tensor,
                workspace: torch.Tensor, stream=None):
    _check("kvd_decode_attn", lib().kvd_decode_attn(
        cache.ref(), _ptr(q), int(q.shape[1]), float(softmax_scale), _ptr(sel_idx),
        _ptr(sel_cnt), int(max_sel), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(q, stream)))


def decode_attn_static(cache: KVCache, q: torch.Tensor, softmax_scale: float,
                       sel_idx: torch.Tensor, sel_cnt: torch.Tensor, max_sel: int,
                       out: torch.Tensor, stream=None):
    """decode_attn with no workspace: the scratch is a fixed array inside the
    library, shared by every call on the device (calls must not overlap)."""
    _check("kvd_decode_attn_static", lib().kvd_decode_attn_static(
        cache.ref(), _ptr(q), int(q.shape[1]), float(softmax_scale), _ptr(sel_idx),
        _ptr(sel_cnt), int(max_sel), _ptr(out), _stream(q, stream)))


def decode_attn_sv(cache: KVCache, q: torch.Tensor, softmax_scale: float, sel_idx,
                   sel_cnt, max_sel: int, sparse_v_eps: float, out: torch.Tensor,
                   workspace: torch.Tensor, stream=None):
    """decode_attn with sparse-V in eps mode; sel_idx None attends every block."""
    _check("kvd_decode_attn_sv", lib().kvd_decode_attn_sv(
        cache.ref(), _ptr(q), int(q.shape[1]), float(softmax_scale), _ptr(sel_idx),
        _ptr(sel_cnt), int(max_sel), float(sparse_v_eps), _ptr(out), _ptr(workspace),
        workspace.numel(), _stream(q, stream)))


def select_blocks_per_head(cache: KVCache, q: torch.Tensor, k_sel: int, sink_tokens: int,
                           recent_tokens: int, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                           workspace: torch.Tensor, stream=None):
    """Selection per query head: sel_idx [B, H, max_seq // 64], sel_cnt [B, H] int32."""
    _check("kvd_select_blocks_per_head", lib().kvd_select_blocks_per_head(
        cache.ref(), _ptr(q), int(q.shape[1]), int(k_sel), int(sink_tokens),
        int(recent_tokens), _ptr(sel_idx), _ptr(sel_cnt), _ptr(workspace), workspace.numel(),
        _stream(q, stream)))


def decode_attn_per_head(cache: KVCache, q: torch.Tensor, softmax_scale: float, sel_idx,
                         sel_cnt, max_sel: int, out: torch.Tensor, workspace: torch.Tensor,
                         stream=None):
    """decode_attn over lists per query head (select_blocks_per_head's rows)."""
    _check("kvd_decode_attn_per_head", lib().kvd_decode_attn_per_head(
        cache.ref(), _ptr(q), int(q.shape[1]), float(softmax_scale), _ptr(sel_idx),
        _ptr(sel_cnt), int(max_sel), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(q, stream)))


def decode_attn_tail(cache: KVCache, q: torch.Tensor, softmax_scale: float, sel_idx, sel_cnt,
                     max_sel: int, out: torch.Tensor, workspace: torch.Tensor, stream=None):
    """decode_attn plus the moment tail of every block the lists leave out
    (needs a cache made with moments=True)."""
    _check("kvd_decode_attn_tail", lib().kvd_decode_attn_tail(
        cache.ref(), _ptr(q), int(q.shape[1]), float(softmax_scale), _ptr(sel_idx),
        _ptr(sel_cnt), int(max_sel), _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(q, stream)))


def decode_attn_dense(cache: KVCache, q: torch.Tensor, softmax_scale: float, out: torch.Tensor,
                      workspace: torch.Tensor, stream=None):
    _check("kvd_decode_attn_dense", lib().kvd_decode_attn_dense(
        cache.ref(), _ptr(q), int(q.shape[1]), float(softmax_scale), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(q, stream)))


def decode_step(cache: KVCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                softmax_scale: float, k_sel: int, sink_tokens: int, recent_tokens: int,
                out: torch.Tensor, workspace: torch.Tensor, sel_idx=None, sel_cnt=None,
                stream=None):
    _check("kvd_decode_step", lib().kvd_decode_step(
        cache.ref(), _ptr(q), _ptr(k_new), _ptr(v_new), int(q.shape[1]), float(softmax_scale),
        k_sel, sink_tokens, recent_tokens, _ptr(sel_idx), _ptr(sel_cnt), _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(workspace, stream)))


def decode_step_host(cache: KVCache, q_host: torch.Tensor, k_new_host: torch.Tensor,
                     v_new_host: torch.Tensor, softmax_scale: float, k_sel: int,
                     sink_tokens: int, recent_tokens: int, out_host: torch.Tensor,
                     workspace: torch.Tensor, sel_idx=None, sel_cnt=None, stream=None):
    """Host (ideally pinned) q/k_new/v_new in, host out; synchronize before reading out."""
    _check("kvd_decode_step_host", lib().kvd_decode_step_host(
        cache.ref(), _ptr(q_host), _ptr(k_new_host), _ptr(v_new_host), int(q_host.shape[1]),
        float(softmax_scale), k_sel, sink_tokens, recent_tokens, _ptr(sel_idx), _ptr(sel_cnt),
        _ptr(out_host), _ptr(workspace), workspace.numel(), _stream(workspace, stream)))


def debug_qk_int8(cache: KVCache, q: torch.Tensor, dots: torch.Tensor, q_codes: torch.Tensor,
                  q_scales: torch.Tensor, stream=None):
    _check("kvd_debug_qk_int8", lib().kvd_debug_qk_int8(
        cache.ref(), _ptr(q), int(q.shape[1]), _ptr(dots), _ptr(q_codes), _ptr(q_scales),
        _stream(q, stream)))


def debug_wait_timeout(status: torch.Tensor, limit_us: int, stream=None):
    """Run the bounded-wait path on a wait that nothing ends (status: int32 [1])."""
    _check("kvd_debug_wait_timeout", lib().kvd_debug_wait_timeout(
        _ptr(status), int(limit_us), _stream(status, stream)))


MARK_SLOTS = 16
MARK_CTAS = 4096
MARK_KINDS = 3


def debug_stage_marks(marks: Optional[torch.Tensor]):
    """Give the library a device buffer for stage marks (int64, at least
    MARK_KINDS * MARK_CTAS * MARK_SLOTS elements), or None to stop recording.
    Raises KvdError (UNSUPPORTED) unless the library was built with marks."""
    n = 0 if marks is None else marks.numel() * marks.element_size()
    _check("kvd_debug_stage_marks", lib().kvd_debug_stage_marks(_ptr(marks), n))


def debug_scores(cache: KVCache, q: torch.Tensor, ub: torch.Tensor, stream=None):
    _check("kvd_debug_scores", lib().kvd_debug_scores(
        cache.ref(), _ptr(q), int(q.shape[1]), _ptr(ub), _stream(q, stream)))


# ------------------------------------------- positions, norms, paged cache ---
_X = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def _heads(t: Optional[torch.Tensor]):
    """kvd_heads of rows [n_tokens, n_heads, head_dim]; only the token stride is free."""
    if t is None:
        return None
    x = _X.get(t.dtype)
    shape = t.shape
    if x is None or len(shape) != 3:
        raise ValueError("rows are [n_tokens, n_heads, head_dim] of float16, bfloat16 or float32")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d != 1) or (s1 != d and h != 1):
        raise ValueError("the heads of a token must be dense")
    return HeadsStruct(t.data_ptr(), s0 if n > 1 else h * d, x, h)


def _int32(t: torch.Tensor, n: int, name: str):
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} is an int32 tensor [{n}]")
    if n > 1 and t.stride()[0] != 1:
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _weight(t: Optional[torch.Tensor], d: int):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != d:
        raise ValueError("a norm weight is a float32 tensor [head_dim]")
    if t.stride()[0] != 1:
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _one_device(index: int, *tensors):
    """All tensors of a call (absent ones None) on CUDA device `index`."""
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("the tensors of a call must be on one device")


def _call(name: str, index: int, stream, fn, *args):
    """The library's call with its device current (it launches there), on the given
    stream or the device's current one."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        raise KvdError(name, rc)


class RopeTable:
    """Rotation of the first rot_dim channels: frequencies on the device and the
    descriptor that points at them.  See rope_table."""

    def __init__(self, freqs: torch.Tensor, rot_dim: int, interleaved: bool, mscale: float):
        self.freqs, self.rot_dim, self.interleaved, self.mscale = freqs, rot_dim, interleaved, mscale
        self.s = RopeStruct(freqs.data_ptr(), rot_dim, int(interleaved), mscale, 0)

    def ref(self):
        return C.byref(self.s)


def rope_table(rot_dim: int, base: float = 10000.0, interleaved: bool = False,
               scaling: str = "none", factor: float = 1.0, orig_len: float = 0.0,
               low: float = 0.0, high: float = 0.0, device="cuda") -> RopeTable:
    """The angles per position of a model's rotation, made once.

    interleaved: pairs (2i, 2i+1), else (i, i + rot_dim/2).  scaling: "none",
    "linear", "ntk", "yarn" or "bands" (kvd_rope_scaling), with the context's
    stretch `factor`, the trained length orig_len and, for the last two, the
    turns in orig_len below which a channel is stretched in full (low) and above
    which it is kept (high); 0 and 0 take the usual ones.  "yarn" multiplies cosines
    and sines by 0.1 ln(factor) + 1 (t.mscale); for a model that puts its factor into
    the softmax scale instead take RopeTable(t.freqs, t.rot_dim, t.interleaved, 1.0)."""
    if scaling not in SCALINGS:
        raise ValueError(f"scaling is one of {sorted(SCALINGS)}")
    words = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.int64)
    m = C.c_float()
    _check("kvd_rope_freqs", lib().kvd_rope_freqs(
        int(rot_dim), float(base), SCALINGS[scaling], float(factor), float(orig_len), float(low),
        float(high), _ptr(words), C.byref(m)))
    return RopeTable(words.to(device), int(rot_dim), bool(interleaved), m.value)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                 rope: Optional[RopeTable], q_out: torch.Tensor, k_out: Optional[torch.Tensor],
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, stream=None):
    """Per-head RMS norm (with a weight) and rotation (with a table) of
    q [T, H, D] and k [T, Hkv, D] into q_out and k_out; positions int32 [T].
    Any of float16, bfloat16 and float32 in, and out; in place too."""
    T, _, D = q.shape
    if q_out.shape != q.shape or (k is not None and (k_out is None or k_out.shape != k.shape or
                                                     k.shape[0] != T or k.shape[2] != D)):
        raise ValueError("outputs have their inputs' shapes, and q and k as many tokens and channels")
    d = q.get_device()
    _one_device(d, k, positions, q_out, k_out, q_weight, k_weight,
                None if rope is None else rope.freqs)
    _call("kvd_qk_norm_rope", d, stream, lib().kvd_qk_norm_rope, _heads(q), _heads(q_out),
          _heads(k), _heads(k_out), T, D,
          None if positions is None else _int32(positions, T, "positions"),
          None if rope is None else rope.s, _weight(q_weight, D), _weight(k_weight, D), eps)


class PagedKVCache:
    """A pool of pages, each sequence's table of them, and the C descriptor.

    k, v        [n_pages, Hkv, page_size, D] float16, bfloat16 or int8 codes; D 64 or 128
    k_scale     [n_pages, Hkv, page_size] float32 (int8); same for v_scale
    page_table  [batch, max_pages] int32: the page of each run of page_size tokens
    seq_lens    [batch] int32: tokens of each sequence, those of the current call
                counted; the caller advances it (once a step, for all layers)
    status      [1] int32 device word for values out of range
    len         at least the largest of seq_lens (host; sizes the grids)
    """

    def __init__(self, dtype: int, batch: int, n_pages: int, n_kv_heads: int, page_size: int,
                 max_pages: int, head_dim: int = HEAD_DIM, device="cuda",
                 tensors: Optional[dict] = None):
        self.dtype, self.batch, self.n_pages, self.n_kv_heads = dtype, batch, n_pages, n_kv_heads
        self.page_size, self.max_pages, self.head_dim = page_size, max_pages, head_dim
        dev = torch.device(device)
        t = dict(tensors) if tensors is not None else {}
        kvt = {F16: torch.float16, BF16: torch.bfloat16}.get(dtype, torch.int8)
        rows = (n_pages, n_kv_heads, page_size)
        want = {"k": (rows + (head_dim,), kvt), "v": (rows + (head_dim,), kvt),
                "page_table": ((batch, max_pages), torch.int32),
                "seq_lens": ((batch,), torch.int32), "status": ((1,), torch.int32)}
        if dtype == INT8:
            want["k_scale"] = want["v_scale"] = (rows, torch.float32)
        for name, (shape, kind) in want.items():
            if name not in t:
                zero = name in ("page_table", "seq_lens", "status")
                t[name] = (torch.zeros if zero else torch.empty)(shape, dtype=kind, device=dev)
            elif tuple(t[name].shape) != shape or t[name].dtype != kind:
                raise ValueError(f"{name} is {kind} of shape {shape}")
        self.t = t
        self.device = t["k"].device
        _one_device(t["k"].get_device(), *t.values())
        self.s = PagedCacheStruct(dtype, batch, n_kv_heads, head_dim, n_pages, page_size,
                                  max_pages, 0, *(_ptr(t.get(n)) for n in (
                                      "k", "v", "k_scale", "v_scale", "page_table", "seq_lens",
                                      "status")))

    @classmethod
    def over(cls, cache: KVCache, seq_lens: Optional[torch.Tensor] = None) -> "PagedKVCache":
        """A float16 or int8 KVCache as a paged one, one page a sequence, over the
        same memory: seq_lens (default: len for each) counts the tokens to attend."""
        if cache.dtype not in (F16, INT8):
            raise KvdError("PagedKVCache.over", 2)
        dev = cache.t["k"].device
        t = {n: cache.t[n] for n in ("k", "v", "k_scale", "v_scale", "status") if n in cache.t}
        t["page_table"] = torch.arange(cache.batch, dtype=torch.int32, device=dev).view(-1, 1)
        t["seq_lens"] = seq_lens if seq_lens is not None else torch.full(
            (cache.batch,), cache.len, dtype=torch.int32, device=dev)
        p = cls(cache.dtype, cache.batch, cache.batch, cache.n_kv_heads, cache.max_seq, 1,
                head_dim=cache.head_dim, device=dev, tensors=t)
        p.len = cache.len
        return p

    @property
    def len(self) -> int:
        return self.s.len

    @len.setter
    def len(self, n: int):
        self.s.len = int(n)

    def __getattr__(self, name):
        t = self.__dict__.get("t")
        if t is not None and name in t:
            return t[name]
        raise AttributeError(name)

    def ref(self):
        return C.byref(self.s)

    def device_status(self) -> int:
        return int(self.t["status"].item())


def paged_workspace_bytes(cache: PagedKVCache, n_heads: int, n_tokens: int, max_new: int) -> int:
    with torch.cuda.device(cache.device):
        return int(lib().kvd_paged_workspace_bytes(cache.ref(), n_heads, n_tokens, max_new))


def make_paged_workspace(cache: PagedKVCache, n_heads: int, n_tokens: int,
                         max_new: int) -> torch.Tensor:
    """A zero-filled workspace for paged_attn calls of up to n_tokens new tokens, up to
    max_new a sequence.  Calls that may overlap on the GPU need one each; after a wait
    that ran out (KVD_ERR_TIMEOUT in the device status) it has to be zeroed."""
    n = paged_workspace_bytes(cache, n_heads, n_tokens, max_new)
    if n == 0:
        raise KvdError("kvd_paged_workspace_bytes", 1)
    return torch.zeros(n, dtype=torch.uint8, device=cache.device)


def paged_append(cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                 rope: Optional[RopeTable] = None, k_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 stream=None):
    """Rows [starts[b], starts[b+1]) of k, v [T, Hkv, D] to sequence b's last positions,
    the keys normed and rotated on the way, and q [T, H, D] with them into q_out."""
    T, _, D = k.shape
    if v.shape != k.shape or D != cache.head_dim:
        raise ValueError("k and v are [n_tokens, n_kv_heads, head_dim]")
    if q is not None and (q_out is None or q_out.shape != q.shape or q.shape[0] != T or
                          q.shape[2] != D):
        raise ValueError("q and q_out are [n_tokens, n_heads, head_dim]")
    d = k.get_device()
    _one_device(d, cache.t["k"], v, starts, k_weight, q, q_out, q_weight,
                None if rope is None else rope.freqs)
    _call("kvd_paged_append", d, stream, lib().kvd_paged_append, cache.s, _heads(k), _heads(v), T,
          _int32(starts, cache.batch + 1, "starts"), None if rope is None else rope.s,
          _weight(k_weight, D), _heads(q), _heads(q_out), _weight(q_weight, D), eps)


def _lse(t: Optional[torch.Tensor], n: int, h: int):
    if t is None:
        return None
    if t.dtype != torch.float32 or tuple(t.shape) != (n, h):
        raise ValueError("lse is a float32 tensor [n_tokens, n_heads]")
    return _ptr(t)


def paged_attn(cache: PagedKVCache, q: torch.Tensor, starts: torch.Tensor, max_new: int,
               softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor, window: int = 0,
               stream=None, lse: Optional[torch.Tensor] = None):
    """Causal attention of rows [starts[b], starts[b+1]) of q [T, H, D], sequence b's last
    tokens, over its pages (with a window: the last `window` keys), into out [T, H, D].
    lse (float32 [T, H]): receives the logarithm of each row's sum of exponentials."""
    T, H, D = q.shape
    if out.shape != q.shape or D != cache.head_dim:
        raise ValueError("q and out are [n_tokens, n_heads, head_dim]")
    d = q.get_device()
    _one_device(d, cache.t["k"], starts, out, workspace, lse)
    args = (cache.s, _heads(q), T, _int32(starts, cache.batch + 1, "starts"), max_new,
            softmax_scale, window, _heads(out))
    ws = (_ptr(workspace), workspace.numel() * workspace.element_size())
    if lse is None:
        _call("kvd_paged_attn", d, stream, lib().kvd_paged_attn, *args, *ws)
    else:
        _call("kvd_paged_attn_lse", d, stream, lib().kvd_paged_attn_lse, *args, _lse(lse, T, H), *ws)


# ------------------------------------------ latent rows, weights, eviction ---
class LatentCache:
    """A pool of pages of rows that all query heads share, and the C descriptor.

    rows        [n_pages, page_size, rank + rope_dim] float16 or bfloat16: a token's normed
                latent vector, then the rotated part of its key
    page_table, seq_lens, status, len: as PagedKVCache
    """

    def __init__(self, dtype: int, batch: int, n_pages: int, page_size: int, max_pages: int,
                 rank: int = 512, rope_dim: int = 64, device="cuda",
                 tensors: Optional[dict] = None):
        self.dtype, self.batch, self.n_pages = dtype, batch, n_pages
        self.page_size, self.max_pages, self.rank, self.rope_dim = page_size, max_pages, rank, rope_dim
        dev = torch.device(device)
        t = dict(tensors) if tensors is not None else {}
        kind = {F16: torch.float16, BF16: torch.bfloat16}.get(dtype)
        if kind is None:
            raise KvdError("LatentCache", 2)
        want = {"rows": ((n_pages, page_size, rank + rope_dim), kind),
                "page_table": ((batch, max_pages), torch.int32),
                "seq_lens": ((batch,), torch.int32), "status": ((1,), torch.int32)}
        for name, (shape, x) in want.items():
            if name not in t:
                t[name] = (torch.empty if name == "rows" else torch.zeros)(shape, dtype=x, device=dev)
            elif tuple(t[name].shape) != shape or t[name].dtype != x:
                raise ValueError(f"{name} is {x} of shape {shape}")
        self.t = t
        self.device = t["rows"].device
        _one_device(t["rows"].get_device(), *t.values())
        self.s = LatentCacheStruct(dtype, batch, rank, rope_dim, n_pages, page_size, max_pages, 0,
                                   *(_ptr(t[n]) for n in ("rows", "page_table", "seq_lens", "status")))

    @property
    def len(self) -> int:
        return self.s.len

    @len.setter
    def len(self, n: int):
        self.s.len = int(n)

    def __getattr__(self, name):
        t = self.__dict__.get("t")
        if t is not None and name in t:
            return t[name]
        raise AttributeError(name)

    def ref(self):
        return C.byref(self.s)

    def device_status(self) -> int:
        return int(self.t["status"].item())


def _part_strides(t: torch.Tensor, name: str):
    """Token and head strides of head parts [n_tokens, n_heads, channels], and the two counts."""
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"the channels of a head of {name} must be dense")
    if h == 1:
        s1 = d
    return n, h, (s0 if n > 1 else h * s1), s1


def latent_append(cache: LatentCache, c: torch.Tensor, k_pe: torch.Tensor, starts: torch.Tensor,
                  rope: Optional[RopeTable] = None, c_weight: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, q_pe: Optional[torch.Tensor] = None,
                  q_out: Optional[torch.Tensor] = None, stream=None):
    """Rows [starts[b], starts[b+1]) of the latents c [T, rank] (normed with c_weight) and the
    shared key parts k_pe [T, rope_dim] (rotated) to sequence b's last positions.  q_pe
    [T, H, rope_dim], rotated too, goes to the last channels of q_out [T, H, rank + rope_dim],
    whose others (the absorbed part) are not touched."""
    T, R = c.shape
    n, P = k_pe.shape
    x = _X.get(c.dtype)
    if R != cache.rank or P != cache.rope_dim or n != T or x is None or k_pe.dtype != c.dtype:
        raise ValueError("c and k_pe are [n_tokens, rank] and [n_tokens, rope_dim] of one type: "
                         "float16, bfloat16 or float32")
    c0, c1 = c.stride()
    k0, k1 = k_pe.stride()
    if c1 != 1 or k1 != 1:
        raise ValueError("the channels of a token must be dense")
    q = to = None
    if q_pe is not None:
        if q_out is None or q_pe.dim() != 3 or q_out.dim() != 3:
            raise ValueError("q_pe and q_out are given together, [n_tokens, n_heads, ..]")
        n, h, q0, q1 = _part_strides(q_pe, "q_pe")
        m, k, o0, o1 = _part_strides(q_out, "q_out")
        y = _X.get(q_out.dtype)
        if n != T or m != T or k != h or q_pe.shape[2] != P or q_out.shape[2] != R + P or \
                q_pe.dtype != c.dtype or y is None:
            raise ValueError("q_pe is [n_tokens, n_heads, rope_dim], q_out [n_tokens, n_heads, "
                             "rank + rope_dim]")
        q = PartsStruct(q_pe.data_ptr(), q0, q1, x, h)
        to = PartsStruct(q_out.data_ptr() + R * (4 if y == 2 else 2), o0, o1, y, h)
    elif q_out is not None:
        raise ValueError("q_pe and q_out are given together")
    d = c.get_device()
    _one_device(d, cache.t["rows"], k_pe, starts, c_weight, q_pe, q_out,
                None if rope is None else rope.freqs)
    _call("kvd_latent_append", d, stream, lib().kvd_latent_append, cache.s,
          HeadsStruct(c.data_ptr(), c0 if T > 1 else R, x, 1),
          HeadsStruct(k_pe.data_ptr(), k0 if T > 1 else P, x, 1), T,
          _int32(starts, cache.batch + 1, "starts"), None if rope is None else rope.s,
          _weight(c_weight, R), q, to, eps)


def latent_workspace_bytes(cache: LatentCache, n_heads: int, n_tokens: int, max_new: int) -> int:
    with torch.cuda.device(cache.device):
        return int(lib().kvd_latent_workspace_bytes(cache.ref(), n_heads, n_tokens, max_new))


def make_latent_workspace(cache: LatentCache, n_heads: int, n_tokens: int,
                          max_new: int) -> torch.Tensor:
    """A workspace for latent_attn calls of up to n_tokens new tokens, up to max_new a
    sequence.  Calls that may overlap on the GPU need one each."""
    n = latent_workspace_bytes(cache, n_heads, n_tokens, max_new)
    if n == 0:
        raise KvdError("kvd_latent_workspace_bytes", 1)
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def latent_attn(cache: LatentCache, q: torch.Tensor, starts: torch.Tensor, max_new: int,
                softmax_scale: float, out: torch.Tensor, workspace: torch.Tensor, window: int = 0,
                stream=None, lse: Optional[torch.Tensor] = None):
    """Causal attention of rows [starts[b], starts[b+1]) of q [T, H, rank + rope_dim], sequence
    b's last tokens, over its latent rows, whose first `rank` channels are the values, into
    out [T, H, rank].  lse as for paged_attn."""
    T, H, W = q.shape
    if tuple(out.shape) != (T, H, cache.rank) or W != cache.rank + cache.rope_dim:
        raise ValueError("q is [n_tokens, n_heads, rank + rope_dim], out [n_tokens, n_heads, rank]")
    d = q.get_device()
    _one_device(d, cache.t["rows"], starts, out, workspace, lse)
    _call("kvd_latent_attn", d, stream, lib().kvd_latent_attn, cache.s, _heads(q), T,
          _int32(starts, cache.batch + 1, "starts"), max_new, softmax_scale, window, _heads(out),
          _lse(lse, T, H), _ptr(workspace), workspace.numel() * workspace.element_size())


def _kind(cache):
    """("latent" or "paged", number of KV heads, channels of a key) of a cache in pages."""
    if isinstance(cache, LatentCache):
        return "latent", 1, cache.rank + cache.rope_dim
    return "paged", cache.n_kv_heads, cache.head_dim


def _mass(t: Optional[torch.Tensor], batch: int, heads: int, least: int, name: str):
    """(pointer, stride) of weights [batch, heads, >= least]; rows dense and evenly apart."""
    if t is None:
        return None, 0
    if t.dtype != torch.float32 or t.dim() != 3 or tuple(t.shape[:2]) != (batch, heads) or \
            t.shape[2] < least:
        raise ValueError(f"{name} is a float32 tensor [batch, n_kv_heads, at least {least}]")
    s0, s1, s2 = t.stride()
    if heads == 1:
        s1 = s0 if batch > 1 else t.shape[2]
    if (s2 != 1 and t.shape[2] > 1) or (batch > 1 and s0 != heads * s1):
        raise ValueError(f"the rows of {name} must be dense and evenly apart")
    return t.data_ptr(), s1


def paged_mass(cache, q: torch.Tensor, lse: torch.Tensor, starts: torch.Tensor, max_new: int,
               softmax_scale: float, mass: Optional[torch.Tensor], out: Optional[torch.Tensor] = None,
               decay: float = 1.0, window: int = 0, stream=None):
    """What an attention call's rows weighed each cached token with, added up a KV head:
    out = decay * mass + the sum of weights, new tokens from 0; mass and out float32 [batch,
    Hkv, >= cache.len] (out None: in place).  cache, q, starts, max_new, softmax_scale and
    window are those of the paged_attn or latent_attn call that gave lse."""
    kind, heads, D = _kind(cache)
    T, H, W = q.shape
    if W != D:
        raise ValueError("q is [n_tokens, n_heads, channels of a key]")
    out = mass if out is None else out
    if out is None or (mass is None and decay != 0):
        raise ValueError("without a mass the decay is 0 and out is given")
    at, stride = _mass(mass, cache.batch, heads, cache.len, "mass")
    to, to_stride = _mass(out, cache.batch, heads, cache.len, "out")
    d = q.get_device()
    _one_device(d, cache.t["page_table"], starts, lse, mass, out)
    name = "kvd_latent_mass" if kind == "latent" else "kvd_paged_mass"
    _call(name, d, stream, getattr(lib(), name), cache.s, _heads(q),
          _lse(lse, T, H), T, _int32(starts, cache.batch + 1, "starts"), max_new, softmax_scale,
          window, at, stride, decay, to, to_stride)


def paged_evict(cache, mass: torch.Tensor, keep: int, page_table_out: torch.Tensor,
                kept: torch.Tensor, seq_lens_out: torch.Tensor,
                mass_out: Optional[torch.Tensor] = None, sink: int = 0, recent: int = 0,
                stream=None):
    """Of each sequence and KV head the first `sink` tokens, the last `recent` and those of
    most mass between, `keep` in all (all of a shorter sequence), in order to the pages of
    page_table_out (int32 [batch, columns]; none that the cache's table needs).  kept (int32
    [batch, Hkv, keep]) receives their old indices, seq_lens_out (int32 [batch]) the new
    lengths, mass_out (float32 [batch, Hkv, >= keep]) their masses.  The caller goes on with
    a cache over the new table and lengths.  Keys keep the rotation of their old positions, so
    later tokens are rotated with qk_norm_rope at positions of the caller's and appended without
    rope; a latent cache's k_pe as k_pe[:, None], its q_pe and q as rows of one head, e.g.
    q_pe.flatten(0, 1)[:, None] into q.view(-1, 1, rank + rope_dim)[..., rank:] (q contiguous, a
    position a row).  An attention's window counts places in the cache."""
    kind, heads, _ = _kind(cache)
    if page_table_out.dtype != torch.int32 or page_table_out.dim() != 2 or \
            page_table_out.shape[0] != cache.batch:
        raise ValueError("page_table_out is an int32 tensor [batch, columns]")
    if kept.dtype != torch.int32 or tuple(kept.shape) != (cache.batch, heads, keep):
        raise ValueError("kept is an int32 tensor [batch, n_kv_heads, keep]")
    at, stride = _mass(mass, cache.batch, heads, cache.len, "mass")
    to, to_stride = _mass(mass_out, cache.batch, heads, keep, "mass_out")
    d = mass.get_device()
    _one_device(d, cache.t["page_table"], page_table_out, kept, seq_lens_out, mass_out)
    name = "kvd_latent_evict" if kind == "latent" else "kvd_paged_evict"
    _call(name, d, stream, getattr(lib(), name), cache.s, at, stride,
          keep, sink, recent, _ptr(page_table_out), page_table_out.shape[1], _ptr(kept),
          _int32(seq_lens_out, cache.batch, "seq_lens_out"), to, to_stride)


__all__ = ["F16", "INT8", "Q8_0", "Q4_0", "BF16", "BLOCK", "HEAD_DIM", "KVCache", "KvdError", "CacheStruct", "lib",
           "debug_stage_marks", "MARK_SLOTS", "MARK_CTAS", "MARK_KINDS",
           "workspace_bytes", "make_workspace", "selected_count", "status_string", "kv_append",
           "kv_append_f32", "select_blocks", "decode_attn", "decode_attn_dense", "decode_attn_static",
           "decode_attn_sv", "decode_attn_tail", "select_blocks_per_head",
           "decode_attn_per_head", "decode_step",
           "decode_step_host", "debug_qk_int8", "debug_scores", "debug_wait_timeout", "synth", "EXPORTS",
           "PagedCacheStruct", "HeadsStruct", "RopeStruct", "RopeTable", "rope_table",
           "qk_norm_rope", "PagedKVCache", "paged_workspace_bytes", "make_paged_workspace",
           "paged_append", "paged_attn", "SCALINGS", "LatentCacheStruct", "PartsStruct",
           "LatentCache", "latent_append", "latent_workspace_bytes", "make_latent_workspace",
           "latent_attn", "paged_mass", "paged_evict"]
