"""GB300-native CSA2 sparse attention over an FP4 global KV cache.

Thin Python binding of ``libcsa2.so`` (the C ABI in ``include/csa2.h``).  It
only marshals arguments: torch tensors become device pointers, the current
torch stream becomes the launch stream, and output tensors are created with
torch when the caller passes none.  Every step of the attention path runs in
the library's CUDA kernels; there is no fallback.  If the library has not been
built the import of this module raises.

Function names follow the C ABI (``csa2_index_topk_decode`` ...).  ``Cache``
owns the device buffer of one CSA2 group's global cache and its handle.
"""
from __future__ import annotations

import array
import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# CSA2_DEBUG=1 loads the bounds-checked build (libcsa2_debug.so, built by
# _build.build(debug=True)); otherwise the normal one.
LIB_PATH = os.path.join(_HERE, "libcsa2_debug.so" if os.environ.get("CSA2_DEBUG") == "1"
                        else "libcsa2.so")

CSA2_KV_L32_UE8M0 = 0
CSA2_KV_L16_E4M3 = 1

STATUS = {0: "CSA2_OK", 1: "CSA2_ERR_INVALID_ARG", 2: "CSA2_ERR_UNSUPPORTED",
          3: "CSA2_ERR_CAPACITY", 4: "CSA2_ERR_CUDA", 5: "CSA2_ERR_OOM",
          6: "CSA2_ERR_TIMEOUT", 7: "CSA2_ERR_DEVICE"}


class Csa2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("swa", ctypes.c_int32),
                ("ratio", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("idx_layout", ctypes.c_int32)]


def config(n_heads=64, head_dim=512, idx_heads=32, idx_dim=128, topk=512, swa=128, ratio=1,
           layout=CSA2_KV_L32_UE8M0, idx_layout=0) -> Config:
    """Layer shapes of the V4.1 report, section 4.2.1, as defaults;
    idx_layout 1 keeps the indexer keys in MXFP4 (CSA2_IDX_MXFP4)."""
    return Config(n_heads, head_dim, idx_heads, idx_dim, topk, swa, ratio, layout, idx_layout)


class AttnOpts(ctypes.Structure):
    """csa2_attn_opts_t: attention sink and output RoPE(-i)."""
    _fields_ = [("sink", ctypes.c_void_p), ("rope_pos", ctypes.c_void_p),
                ("rope_out", ctypes.c_int32), ("rope_base", ctypes.c_double),
                ("swa_codes", ctypes.c_void_p), ("swa_rope", ctypes.c_void_p),
                ("swa_scales", ctypes.c_void_p)]


class CacheViews(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("idx_k", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("entry_offset", ctypes.POINTER(ctypes.c_int64)), ("total", ctypes.c_int64),
                ("batch", ctypes.c_int32), ("group", ctypes.c_int32),
                ("idx_codes", ctypes.c_void_p), ("idx_scales", ctypes.c_void_p)]


class TreeStruct(ctypes.Structure):
    """csa2_tree_t."""
    _fields_ = [("n_seqs", ctypes.c_int32), ("seq_ids", ctypes.c_void_p),
                ("n_draft", ctypes.c_void_p), ("pos0", ctypes.c_void_p),
                ("parent", ctypes.c_void_p)]


class TreeLayer(ctypes.Structure):
    """csa2_tree_layer_t: one layer of a drafted tree's readout (_TREE_LAYER
    packs the same fields)."""
    _fields_ = [(f, ctypes.c_void_p) for f in
                ("q", "swa_kv", "draft_kv", "out", "lse", "sink", "swa_codes", "swa_rope",
                 "swa_scales", "draft_codes", "draft_rope", "draft_scales")]


class NormPart(ctypes.Structure):
    """csa2_norm_part_t: one tensor of a norm + rotation call (_NORM_PART packs
    the same fields)."""
    _fields_ = ([(f, ctypes.c_void_p) for f in ("x", "out", "weight", "pos")] +
                [(f, ctypes.c_int64) for f in ("n_tokens", "x_token_stride", "x_head_stride",
                                               "out_token_stride", "out_head_stride")] +
                [(f, ctypes.c_int32) for f in ("n_heads", "dim", "rope_dim", "norm", "x_fp32",
                                               "out_fp32")])


class WindowStruct(ctypes.Structure):
    """csa2_window_t."""
    _fields_ = ([(f, ctypes.c_int32) for f in ("n_seqs", "swa", "n_first", "fp8")] +
                [(f, ctypes.c_void_p) for f in ("rows", "codes", "rope", "scales", "pos", "error")])


class WindowOpts(ctypes.Structure):
    """csa2_window_opts_t."""
    _fields_ = [("sink", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("rope_out", ctypes.c_int32),
                ("rope_base", ctypes.c_double), ("error", ctypes.c_void_p),
                ("wait_cycles", ctypes.c_int64), ("withhold", ctypes.c_int32)]


class VerifyStruct(ctypes.Structure):
    """csa2_verify_t."""
    _fields_ = ([(f, ctypes.c_int32) for f in ("vocab", "fp32")] +
                [(f, ctypes.c_void_p) for f in ("token", "target", "target_root", "draft",
                                                "draft_root")] +
                [("ld", ctypes.c_int64)] +
                [(f, ctypes.c_void_p) for f in ("temperature", "uniform", "noise")] +
                [("noise_ld", ctypes.c_int64)] +
                [(f, ctypes.c_void_p) for f in ("accepted", "next_token")])


_NORM_PART = struct.Struct("@4P5q6i")
_TREE_LAYER = struct.Struct("@12P")
assert _NORM_PART.size == ctypes.sizeof(NormPart)
assert _TREE_LAYER.size == ctypes.sizeof(TreeLayer)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(the CSA2 path has no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    pcfg = ctypes.POINTER(Config)
    sigs = {
        "csa2_version": ([], i32),
        "csa2_status_string": ([i32], ctypes.c_char_p),
        "csa2_cache_bytes": ([pcfg, i32, P], sz),
        "csa2_cache_create": ([pcfg, i32, P, P, sz, P, ctypes.POINTER(P)], i32),
        "csa2_cache_destroy": ([P], i32),
        "csa2_cache_set_index_sms": ([P, i32], i32),
        "csa2_cache_set_wait_limit": ([P, i64], i32),
        "csa2_cache_inject_fault": ([P, i32], i32),
        "csa2_cache_reset": ([P, P], i32),
        "csa2_cache_length": ([P, i32, ctypes.POINTER(i64)], i32),
        "csa2_cache_views": ([P, ctypes.POINTER(CacheViews)], i32),
        "csa2_compress": ([i32, i64, i32, P, P, P, P], i32),
        "csa2_append_entries": ([P, i32, P, P, P, P, P], i32),
        "csa2_append_tokens": ([P, i32, P, P, P, P, P, P, P], i32),
        "csa2_index_workspace_bytes": ([P, i32], sz),
        "csa2_index_scores_decode": ([P, i32, P, P, P, P, i64, P, P], i32),
        "csa2_index_topk_decode": ([P, i32, P, P, P, P, P, P, sz, P], i32),
        "csa2_index_topk_prefill": ([P, i32, i32, i64, P, P, P, P, P, sz, P], i32),
        "csa2_index_topk_decode_static": ([P, i32, P, P, P, P, P, P], i32),
        "csa2_index_topk": ([P, i32, P, P, P, P, P, P, P, sz, P], i32),
        "csa2_index_scores_prefill": ([P, i32, i32, i64, P, P, P, i64, P, P], i32),
        "csa2_index_prefill_workspace_bytes": ([P, i32, i32], sz),
        "csa2_index_scores_decode_bf16": ([P, i32, P, P, P, P, i64, P, P], i32),
        "csa2_topk_bf16": ([i32, P, i64, P, i32, P, P, P, P, sz, P], i32),
        "csa2_index_topk_decode_bf16": ([P, i32, P, P, P, P, P, P, sz, P], i32),
        "csa2_sparse_attn_decode_ex": ([P, i32, P, P, P, P, P, ctypes.c_float, P, P, P, sz, P,
                                        P], i32),
        "csa2_sparse_attn_decode_layers": ([P, i32, i32, P, P, P, P, P, ctypes.c_float, P, P, P, sz,
                                            P, P], i32),
        "csa2_sparse_attn_prefill_ex": ([P, i32, i32, i64, P, P, i64, i64, P, ctypes.c_float, P,
                                         P, P, P], i32),
        "csa2_sparse_attn_prefill_layers": ([P, i32, i32, i32, i64, P, P, i64, i64, P,
                                             ctypes.c_float, P, P, P, P], i32),
        "csa2_swa_fp8_quantise": ([i64, P, P, P, P, P], i32),
        "csa2_hsi_pool_workspace_bytes": ([i32, i64], sz),
        "csa2_hsi_pool": ([i32, P, i64, P, i32, i32, P, P, sz, P], i32),
        "csa2_index_reindex_workspace_bytes": ([P, i32, i32], sz),
        "csa2_index_topk_reindex_decode": ([P, i32, P, P, P, P, i32, P, P, P, sz, P], i32),
        "csa2_topk_workspace_bytes": ([i32, i64], sz),
        "csa2_topk": ([i32, P, i64, P, i32, P, P, P, P, sz, P], i32),
        "csa2_sparse_attn_workspace_bytes": ([P, i32], sz),
        "csa2_sparse_attn_decode": ([P, i32, P, P, P, P, P, ctypes.c_float, P, P, P, sz, P], i32),
        "csa2_sparse_attn_prefill": ([P, i32, i32, i64, P, P, i64, i64, P, ctypes.c_float, P, P,
                                      P], i32),
        "csa2_get_device_error": ([P, P, ctypes.POINTER(i32)], i32),
        "csa2_norm_rope": ([i32, P, ctypes.c_float, ctypes.c_double, P], i32),
        "csa2_tree_paths": ([i32, P, P, P], i32),
        "csa2_index_scores_tree": ([P, P, P, P, P, i64, P, P], i32),
        "csa2_index_topk_tree": ([P, P, P, P, P, P, P, sz, P], i32),
        "csa2_sparse_attn_tree": ([P, P, i32, P, P, P, ctypes.c_float, i32, ctypes.c_double, P,
                                   sz, P], i32),
        "csa2_cache_accept_tree": ([P, P, P, P], i32),
        "csa2_window_reset": ([P, i32, P], i32),
        "csa2_window_append": ([P, i32, P, P, P, P, P, P], i32),
        "csa2_window_read": ([P, i32, P, P, i32, P, P, P, P, P, P], i32),
        "csa2_window_attn_decode": ([P, i32, i32, P, P, P, ctypes.c_float, P, P, P], i32),
        "csa2_window_attn_tree": ([P, P, i32, P, P, P, P, P, ctypes.c_float, P, P, P], i32),
        "csa2_window_accept_tree": ([P, P, P, P, P, P, P, P], i32),
        "csa2_window_attn_prefill": ([i32, i32, i64, P, P, i64, i64, i32, P, i32, ctypes.c_float, P,
                                      P, P], i32),
        "csa2_window_device_error": ([P, P, ctypes.POINTER(i32)], i32),
        "csa2_verify_tree": ([P, P, P], i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = _load()


def _check(st: int, what: str):
    if st != 0:
        raise Csa2Error(st, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None, device: Optional[int] = None):
    """The launch stream; `device`: the current device where the caller has
    it, which spares the lookup."""
    if stream is None and device is not None:
        return torch._C._cuda_getCurrentRawStream(device)
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _i32_array(xs: Optional[Sequence[int]]):
    if xs is None:
        return None
    n = len(xs)
    if n > 8 and isinstance(xs, (list, tuple)):
        try:   # several times faster than one by one
            return (ctypes.c_int32 * n).from_buffer(array.array("i", xs))
        except (TypeError, OverflowError):
            pass
    return (ctypes.c_int32 * n)(*[int(x) for x in xs])


def _i64_array(xs: Sequence[int]):
    return (ctypes.c_int64 * len(xs))(*[int(x) for x in xs])


class Cache:
    """One CSA2 group's global KV cache in a torch-owned device buffer."""

    def __init__(self, cfg: Config, capacity: Sequence[int], device=None, stream=None):
        self.cfg = cfg
        self.batch = len(capacity)
        caps = _i64_array(capacity)
        nbytes = lib.csa2_cache_bytes(ctypes.byref(cfg), self.batch, caps)
        if nbytes == 0:
            raise Csa2Error(1, "csa2_cache_bytes")
        device = torch.device("cuda") if device is None else torch.device(device)
        # the cache at a 256-byte boundary, and behind it 16 bytes: the token
        # workspace of readouts that are given none
        self.buffer = torch.empty(nbytes + 256 + 32, dtype=torch.uint8, device=device)
        self._off = (-self.buffer.data_ptr()) % 256
        self._token = self.buffer.data_ptr() + self._off + (nbytes + 15) // 16 * 16
        self.handle = ctypes.c_void_p()
        _check(lib.csa2_cache_create(ctypes.byref(cfg), self.batch, caps,
                                     ctypes.c_void_p(self.buffer.data_ptr() + self._off),
                                     nbytes, _stream(stream), ctypes.byref(self.handle)),
               "csa2_cache_create")

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            lib.csa2_cache_destroy(h)
            self.handle = None

    def length(self, seq: int) -> int:
        n = ctypes.c_int64()
        _check(lib.csa2_cache_length(self.handle, seq, ctypes.byref(n)), "csa2_cache_length")
        return n.value

    def reset(self, stream=None):
        _check(lib.csa2_cache_reset(self.handle, _stream(stream)), "csa2_cache_reset")

    def set_index_sms(self, n_sms: int):
        """At most n_sms SMs for the indexer's grid (0: all); see
        csa2_cache_set_index_sms."""
        _check(lib.csa2_cache_set_index_sms(self.handle, n_sms), "csa2_cache_set_index_sms")

    def set_wait_limit(self, cycles: int):
        """Bounded-wait limit of this cache's kernels in SM cycles (0: the
        default); see csa2_cache_set_wait_limit."""
        _check(lib.csa2_cache_set_wait_limit(self.handle, cycles), "csa2_cache_set_wait_limit")

    def inject_fault(self, fault: int):
        """0: none; 1: the indexers issue no key loads (tests of the timeout
        path); see csa2_cache_inject_fault."""
        _check(lib.csa2_cache_inject_fault(self.handle, fault), "csa2_cache_inject_fault")

    def views(self) -> dict:
        """codes [total, 256] u8, scales [total, 512/g] u8, idx_k [total, 128]
        bf16, lengths [batch] int32, entry_offset (list), group."""
        v = CacheViews()
        _check(lib.csa2_cache_views(self.handle, ctypes.byref(v)), "csa2_cache_views")
        base = self.buffer.data_ptr()
        total = v.total

        def sl(ptr, nbytes):
            o = ptr - base
            return self.buffer[o:o + nbytes]

        g = v.group
        mx = bool(v.idx_codes)
        return {
            "codes": sl(v.codes, total * 256).view(total, 256),
            "scales": sl(v.scales, total * (512 // g)).view(total, 512 // g),
            "idx_k": None if mx else sl(v.idx_k, total * 256).view(torch.bfloat16).view(total, 128),
            "idx_codes": sl(v.idx_codes, total * 64).view(total, 64) if mx else None,
            "idx_scales": sl(v.idx_scales, total * 4).view(total, 4) if mx else None,
            "lengths": sl(v.lengths, 4 * self.batch).view(torch.int32),
            "entry_offset": [v.entry_offset[i] for i in range(self.batch + 1)],
            "group": g,
        }

    def device_error(self, stream=None) -> int:
        st = ctypes.c_int32()
        _check(lib.csa2_get_device_error(self.handle, _stream(stream), ctypes.byref(st)),
               "csa2_get_device_error")
        return st.value


# ------------------------------------------------------------------ compress / append
def csa2_compress(ratio: int, c_tok: torch.Tensor, z_tok: torch.Tensor,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    t, dim = c_tok.shape
    n_out = t // ratio
    if out is None:
        out = torch.empty(n_out, dim, dtype=torch.float32, device=c_tok.device)
    _check(lib.csa2_compress(ratio, n_out, dim, _ptr(c_tok), _ptr(z_tok), _ptr(out),
                             _stream(stream)), "csa2_compress")
    return out


def csa2_append_entries(cache: Cache, seq_ids: Sequence[int], n_new: Sequence[int],
                        entries: torch.Tensor, idx_k: torch.Tensor, stream=None):
    _check(lib.csa2_append_entries(cache.handle, len(seq_ids), _i32_array(seq_ids),
                                   _i32_array(n_new), _ptr(entries), _ptr(idx_k),
                                   _stream(stream)), "csa2_append_entries")


def csa2_append_tokens(cache: Cache, seq_ids: Sequence[int], n_tok: Sequence[int],
                       c_tok: torch.Tensor, z_tok: torch.Tensor, idx_k: torch.Tensor,
                       entries_out: Optional[torch.Tensor] = None, stream=None):
    _check(lib.csa2_append_tokens(cache.handle, len(seq_ids), _i32_array(seq_ids),
                                  _i32_array(n_tok), _ptr(c_tok), _ptr(z_tok), _ptr(idx_k),
                                  _ptr(entries_out), _stream(stream)), "csa2_append_tokens")


# ------------------------------------------------------------------ indexer + top-k
def csa2_index_workspace_bytes(cache: Cache, n_queries: int) -> int:
    return int(lib.csa2_index_workspace_bytes(cache.handle, n_queries))


def _workspace(nbytes: int, device, workspace):
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    return workspace


def csa2_index_scores_decode(cache: Cache, q_idx: torch.Tensor, w: torch.Tensor,
                             scores: torch.Tensor, seq_ids: Optional[Sequence[int]] = None,
                             key_hist: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """scores: fp32 [n_queries, ld] (ld a multiple of 4, >= every length);
    key_hist: optional int32 [n_queries, 2048] score-key histogram output."""
    _check(lib.csa2_index_scores_decode(cache.handle, q_idx.shape[0], _ptr(q_idx), _ptr(w),
                                        _i32_array(seq_ids), _ptr(scores), scores.shape[1],
                                        _ptr(key_hist), _stream(stream)),
           "csa2_index_scores_decode")
    return scores


def csa2_index_topk_decode(cache: Cache, q_idx: torch.Tensor, w: torch.Tensor,
                           seq_ids: Optional[Sequence[int]] = None,
                           topk_idx: Optional[torch.Tensor] = None,
                           topk_score: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    nq = q_idx.shape[0]
    dev = q_idx.device
    if topk_idx is None:
        topk_idx = torch.empty(nq, cache.cfg.topk, dtype=torch.int32, device=dev)
    ws = _workspace(csa2_index_workspace_bytes(cache, nq), dev, workspace)
    _check(lib.csa2_index_topk_decode(cache.handle, nq, _ptr(q_idx), _ptr(w),
                                      _i32_array(seq_ids), _ptr(topk_idx), _ptr(topk_score),
                                      _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "csa2_index_topk_decode")
    return topk_idx


def csa2_index_topk(cache: Cache, q_idx: torch.Tensor, w: torch.Tensor,
                    seq_of_q: Optional[Sequence[int]], q_pos: Sequence[int],
                    topk_idx: Optional[torch.Tensor] = None,
                    topk_score: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Selection for queries at token positions q_pos of sequences seq_of_q
    (host lists; seq_of_q None: query i reads sequence i)."""
    nq = q_idx.shape[0]
    dev = q_idx.device
    if topk_idx is None:
        topk_idx = torch.empty(nq, cache.cfg.topk, dtype=torch.int32, device=dev)
    ws = _workspace(csa2_index_workspace_bytes(cache, nq), dev, workspace)
    _check(lib.csa2_index_topk(cache.handle, nq, _ptr(q_idx), _ptr(w), _i32_array(seq_of_q),
                               _i64_array(q_pos), _ptr(topk_idx), _ptr(topk_score), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)),
           "csa2_index_topk")
    return topk_idx


def csa2_index_scores_prefill(cache: Cache, seq: int, pos0: int, q_idx: torch.Tensor,
                              w: torch.Tensor, scores: torch.Tensor,
                              key_hist: Optional[torch.Tensor] = None, stream=None):
    """scores: fp32 [n_queries, ld] (ld a multiple of 4, >= the length);
    key_hist: int32 [n_queries, 2048] score-key histograms (bf16 keys)."""
    _check(lib.csa2_index_scores_prefill(cache.handle, seq, q_idx.shape[0], pos0, _ptr(q_idx),
                                         _ptr(w), _ptr(scores), scores.shape[1], _ptr(key_hist),
                                         _stream(stream)), "csa2_index_scores_prefill")
    return scores


def csa2_index_prefill_workspace_bytes(cache: Cache, seq: int, n_queries: int) -> int:
    return int(lib.csa2_index_prefill_workspace_bytes(cache.handle, seq, n_queries))


def csa2_index_topk_prefill(cache: Cache, seq: int, pos0: int, q_idx: torch.Tensor,
                            w: torch.Tensor, topk_idx: Optional[torch.Tensor] = None,
                            topk_score: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    nq = q_idx.shape[0]
    dev = q_idx.device
    if topk_idx is None:
        topk_idx = torch.empty(nq, cache.cfg.topk, dtype=torch.int32, device=dev)
    ws = _workspace(csa2_index_prefill_workspace_bytes(cache, seq, nq), dev, workspace)
    _check(lib.csa2_index_topk_prefill(cache.handle, seq, nq, pos0, _ptr(q_idx), _ptr(w),
                                       _ptr(topk_idx), _ptr(topk_score), _ptr(ws),
                                       ws.numel() * ws.element_size(), _stream(stream)),
           "csa2_index_topk_prefill")
    return topk_idx


def csa2_topk_workspace_bytes(n_rows: int, max_valid: int) -> int:
    return int(lib.csa2_topk_workspace_bytes(n_rows, max_valid))


def csa2_topk(scores: torch.Tensor, n_valid: Sequence[int], k: int,
              idx_out: Optional[torch.Tensor] = None, score_out: Optional[torch.Tensor] = None,
              key_hist: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None):
    rows, ld = scores.shape
    if idx_out is None:
        idx_out = torch.empty(rows, k, dtype=torch.int32, device=scores.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.csa2_topk(rows, _ptr(scores), ld, _i64_array(n_valid), k, _ptr(key_hist),
                         _ptr(idx_out), _ptr(score_out), _ptr(workspace), ws_bytes,
                         _stream(stream)), "csa2_topk")
    return idx_out


# ------------------------------------------------------------------ attention
def csa2_sparse_attn_workspace_bytes(cache: Cache, n_queries: int) -> int:
    return int(lib.csa2_sparse_attn_workspace_bytes(cache.handle, n_queries))


def csa2_sparse_attn_decode(cache: Cache, q: torch.Tensor, swa_kv: Optional[torch.Tensor],
                            topk_idx: torch.Tensor, scale: float,
                            swa_len: Optional[torch.Tensor] = None,
                            seq_ids: Optional[Sequence[int]] = None,
                            out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            sink: Optional[torch.Tensor] = None,
                            rope_pos: Optional[torch.Tensor] = None, rope_base: float = 0.0,
                            swa_fp8=None, stream=None) -> torch.Tensor:
    """workspace=None allocates one of csa2_sparse_attn_workspace_bytes; pass
    an empty tensor to run without (one CTA per query).  sink: fp32 [n_heads]
    per-head sink logits; rope_pos: int64 [n_queries] positions i for the
    output RoPE(-i)."""
    nq = q.shape[0]
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.empty(max(16, csa2_sparse_attn_workspace_bytes(cache, nq)),
                                dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    args = (cache.handle, nq, _i32_array(seq_ids), _ptr(q), _ptr(swa_kv), _ptr(swa_len),
            _ptr(topk_idx), float(scale), _ptr(out), _ptr(lse),
            _ptr(workspace) if ws_bytes else None, ws_bytes)
    if sink is None and rope_pos is None and swa_fp8 is None:
        _check(lib.csa2_sparse_attn_decode(*args, _stream(stream)), "csa2_sparse_attn_decode")
    else:
        f8 = swa_fp8 if swa_fp8 is not None else (None, None, None)
        opts = AttnOpts(_ptr(sink), _ptr(rope_pos), 1 if rope_pos is not None else 0,
                        float(rope_base), _ptr(f8[0]), _ptr(f8[1]), _ptr(f8[2]))
        _check(lib.csa2_sparse_attn_decode_ex(*args, ctypes.byref(opts), _stream(stream)),
               "csa2_sparse_attn_decode_ex")
    return out


def csa2_sparse_attn_decode_layers(cache: Cache, qs: Sequence[torch.Tensor],
                                   swa_kvs: Optional[Sequence[Optional[torch.Tensor]]],
                                   topk_idx: torch.Tensor, scale: float,
                                   outs: Sequence[torch.Tensor],
                                   lses: Optional[Sequence[Optional[torch.Tensor]]] = None,
                                   swa_len: Optional[torch.Tensor] = None,
                                   seq_ids: Optional[Sequence[int]] = None,
                                   workspace: Optional[torch.Tensor] = None,
                                   sinks: Optional[Sequence[Optional[torch.Tensor]]] = None,
                                   rope_pos: Optional[torch.Tensor] = None, rope_base: float = 0.0,
                                   swa_fp8s=None, stream=None):
    """The readout of several layers of a group in one launch (per layer:
    queries, window rows or their FP8 form, sink, outputs); workspace as for
    csa2_sparse_attn_decode."""
    L = len(qs)
    nq = qs[0].shape[0]
    if workspace is None:
        workspace = torch.empty(max(16, csa2_sparse_attn_workspace_bytes(cache, nq)),
                                dtype=torch.uint8, device=qs[0].device)
    ws_bytes = workspace.numel() * workspace.element_size()
    arr = lambda xs: (ctypes.c_void_p * L)(*[_ptr(x) for x in xs])
    swa_arr = arr(swa_kvs) if swa_kvs is not None else None
    lse_arr = arr(lses) if lses is not None else None
    keep = []
    opts_arr = None
    if sinks is not None or rope_pos is not None or swa_fp8s is not None:
        ptrs = []
        for l in range(L):
            f8 = swa_fp8s[l] if swa_fp8s is not None and swa_fp8s[l] is not None else (None, None, None)
            o = AttnOpts(_ptr(sinks[l] if sinks is not None else None), _ptr(rope_pos),
                         1 if rope_pos is not None else 0, float(rope_base),
                         _ptr(f8[0]), _ptr(f8[1]), _ptr(f8[2]))
            keep.append(o)
            ptrs.append(ctypes.cast(ctypes.pointer(o), ctypes.c_void_p))
        opts_arr = (ctypes.c_void_p * L)(*ptrs)
    _check(lib.csa2_sparse_attn_decode_layers(cache.handle, L, nq, _i32_array(seq_ids), arr(qs),
                                              swa_arr, _ptr(swa_len), _ptr(topk_idx),
                                              float(scale), arr(outs), lse_arr,
                                              _ptr(workspace) if ws_bytes else None, ws_bytes,
                                              opts_arr, _stream(stream)),
           "csa2_sparse_attn_decode_layers")
    return outs


def csa2_sparse_attn_prefill(cache: Cache, seq: int, pos0: int, q: torch.Tensor,
                             swa_kv: Optional[torch.Tensor], swa_pos0: int,
                             topk_idx: torch.Tensor, scale: float,
                             out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None,
                             sink: Optional[torch.Tensor] = None, rope_out: bool = False,
                             rope_base: float = 0.0, swa_fp8=None, stream=None) -> torch.Tensor:
    """rope_out: rotate the last 64 output channels by RoPE(-(pos0 + i));
    swa_fp8: (codes, rope, scales) of csa2_swa_fp8_quantise instead of
    swa_kv."""
    nq = q.shape[0]
    if out is None:
        out = torch.empty_like(q)
    n_rows = swa_fp8[0].shape[0] if swa_fp8 is not None else (
        swa_kv.shape[0] if swa_kv is not None else 0)
    args = (cache.handle, seq, nq, pos0, _ptr(q), _ptr(swa_kv), swa_pos0, n_rows,
            _ptr(topk_idx), float(scale), _ptr(out), _ptr(lse))
    if sink is None and not rope_out and swa_fp8 is None:
        _check(lib.csa2_sparse_attn_prefill(*args, _stream(stream)), "csa2_sparse_attn_prefill")
    else:
        f8 = swa_fp8 if swa_fp8 is not None else (None, None, None)
        opts = AttnOpts(_ptr(sink), None, 1 if rope_out else 0, float(rope_base),
                        _ptr(f8[0]), _ptr(f8[1]), _ptr(f8[2]))
        _check(lib.csa2_sparse_attn_prefill_ex(*args, ctypes.byref(opts), _stream(stream)),
               "csa2_sparse_attn_prefill_ex")
    return out


def csa2_sparse_attn_prefill_layers(cache: Cache, seq: int, pos0: int,
                                    qs: Sequence[torch.Tensor],
                                    swa_kvs: Optional[Sequence[Optional[torch.Tensor]]],
                                    swa_pos0: int, topk_idx: torch.Tensor, scale: float,
                                    outs: Sequence[torch.Tensor],
                                    lses: Optional[Sequence[Optional[torch.Tensor]]] = None,
                                    sinks: Optional[Sequence[Optional[torch.Tensor]]] = None,
                                    rope_out: bool = False, rope_base: float = 0.0,
                                    swa_fp8s=None, stream=None):
    """The prefill readout of several layers of a group in one launch (per
    layer: queries, window rows or their FP8 form, sink, outputs)."""
    L = len(qs)
    nq = qs[0].shape[0]
    n_rows = 0
    for l in range(L):
        if swa_fp8s is not None and swa_fp8s[l] is not None:
            n_rows = swa_fp8s[l][0].shape[0]
        elif swa_kvs is not None and swa_kvs[l] is not None:
            n_rows = swa_kvs[l].shape[0]
    arr = lambda xs: (ctypes.c_void_p * L)(*[_ptr(x) for x in xs])
    swa_arr = arr(swa_kvs) if swa_kvs is not None else None
    lse_arr = arr(lses) if lses is not None else None
    keep = []
    opts_arr = None
    if sinks is not None or rope_out or swa_fp8s is not None:
        ptrs = []
        for l in range(L):
            f8 = swa_fp8s[l] if swa_fp8s is not None and swa_fp8s[l] is not None else (None, None, None)
            o = AttnOpts(_ptr(sinks[l] if sinks is not None else None), None,
                         1 if rope_out else 0, float(rope_base),
                         _ptr(f8[0]), _ptr(f8[1]), _ptr(f8[2]))
            keep.append(o)
            ptrs.append(ctypes.cast(ctypes.pointer(o), ctypes.c_void_p))
        opts_arr = (ctypes.c_void_p * L)(*ptrs)
    _check(lib.csa2_sparse_attn_prefill_layers(cache.handle, seq, L, nq, pos0, arr(qs), swa_arr,
                                               swa_pos0, n_rows, _ptr(topk_idx), float(scale),
                                               arr(outs), lse_arr, opts_arr, _stream(stream)),
           "csa2_sparse_attn_prefill_layers")
    return outs


# ------------------------------------------------------------------ hierarchical sparse indexer
def csa2_hsi_pool(scores: torch.Tensor, n_valid: Sequence[int], max_blocks: int = 2048,
                  block: int = 8, pool_blocks: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """scores: fp32 [rows, ld] of a Full layer; returns int32 [rows, max_blocks]
    kept block indices (ascending, -1 padded)."""
    rows, ld = scores.shape
    if pool_blocks is None:
        pool_blocks = torch.empty(rows, max_blocks, dtype=torch.int32, device=scores.device)
    workspace = _workspace(int(lib.csa2_hsi_pool_workspace_bytes(rows, max(n_valid, default=0))),
                           scores.device, workspace)
    _check(lib.csa2_hsi_pool(rows, _ptr(scores), ld, _i64_array(n_valid), block, max_blocks,
                             _ptr(pool_blocks), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)),
           "csa2_hsi_pool")
    return pool_blocks


def csa2_index_topk_reindex_decode(cache: Cache, q_idx: torch.Tensor, w: torch.Tensor,
                                   pool_blocks: torch.Tensor,
                                   seq_ids: Optional[Sequence[int]] = None,
                                   topk_idx: Optional[torch.Tensor] = None,
                                   topk_score: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None,
                                   stream=None) -> torch.Tensor:
    """Reindex-layer top-k inside each query's pool (pool_blocks from
    csa2_hsi_pool, one row per query); returns int32 [n_queries, topk]."""
    nq, max_blocks = pool_blocks.shape
    if topk_idx is None:
        topk_idx = torch.empty(nq, cache.cfg.topk, dtype=torch.int32, device=q_idx.device)
    workspace = _workspace(int(lib.csa2_index_reindex_workspace_bytes(cache.handle, nq, max_blocks)),
                           q_idx.device, workspace)
    _check(lib.csa2_index_topk_reindex_decode(cache.handle, nq, _ptr(q_idx), _ptr(w),
                                              _i32_array(seq_ids), _ptr(pool_blocks), max_blocks,
                                              _ptr(topk_idx), _ptr(topk_score), _ptr(workspace),
                                              workspace.numel() * workspace.element_size(),
                                              _stream(stream)),
           "csa2_index_topk_reindex_decode")
    return topk_idx


# ------------------------------------------------------------------ bf16-rounded scores
def csa2_index_scores_decode_bf16(cache: Cache, q_idx: torch.Tensor, w: torch.Tensor,
                                  scores: torch.Tensor, seq_ids: Optional[Sequence[int]] = None,
                                  key_hist: Optional[torch.Tensor] = None,
                                  stream=None) -> torch.Tensor:
    """scores: bf16 (or int16) [n_queries, ld], ld a multiple of 8."""
    _check(lib.csa2_index_scores_decode_bf16(cache.handle, q_idx.shape[0], _ptr(q_idx), _ptr(w),
                                             _i32_array(seq_ids), _ptr(scores), scores.shape[1],
                                             _ptr(key_hist), _stream(stream)),
           "csa2_index_scores_decode_bf16")
    return scores


def csa2_topk_bf16(scores: torch.Tensor, n_valid: Sequence[int], k: int,
                   idx_out: Optional[torch.Tensor] = None,
                   score_out: Optional[torch.Tensor] = None,
                   key_hist: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    rows, ld = scores.shape
    if idx_out is None:
        idx_out = torch.empty(rows, k, dtype=torch.int32, device=scores.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.csa2_topk_bf16(rows, _ptr(scores), ld, _i64_array(n_valid), k, _ptr(key_hist),
                              _ptr(idx_out), _ptr(score_out), _ptr(workspace), nbytes,
                              _stream(stream)),
           "csa2_topk_bf16")
    return idx_out


def csa2_index_topk_decode_bf16(cache: Cache, q_idx: torch.Tensor, w: torch.Tensor,
                                seq_ids: Optional[Sequence[int]] = None,
                                topk_idx: Optional[torch.Tensor] = None,
                                topk_score: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    nq = q_idx.shape[0]
    dev = q_idx.device
    if topk_idx is None:
        topk_idx = torch.empty(nq, cache.cfg.topk, dtype=torch.int32, device=dev)
    ws = _workspace(csa2_index_workspace_bytes(cache, nq), dev, workspace)
    _check(lib.csa2_index_topk_decode_bf16(cache.handle, nq, _ptr(q_idx), _ptr(w),
                                           _i32_array(seq_ids), _ptr(topk_idx), _ptr(topk_score),
                                           _ptr(ws), ws.numel() * ws.element_size(),
                                           _stream(stream)),
           "csa2_index_topk_decode_bf16")
    return topk_idx


# ------------------------------------------------------------------ FP8 window rows
def csa2_swa_fp8_quantise(rows: torch.Tensor, stream=None):
    """bf16 rows [..., 512] -> (codes u8 [n, 448], rope bf16 [n, 64],
    scales u8 [n, 8]) with n the number of rows."""
    r = rows.reshape(-1, 512)
    n = r.shape[0]
    codes = torch.empty(n, 448, dtype=torch.uint8, device=rows.device)
    rope = torch.empty(n, 64, dtype=torch.bfloat16, device=rows.device)
    scales = torch.empty(n, 8, dtype=torch.uint8, device=rows.device)
    _check(lib.csa2_swa_fp8_quantise(n, _ptr(r), _ptr(codes), _ptr(rope), _ptr(scales),
                                     _stream(stream)), "csa2_swa_fp8_quantise")
    return codes, rope, scales


# ------------------------------------------------------------------ norms and rotation
def _shaped(t: torch.Tensor, shape, dtype, what: str, dev: int):
    """Device pointer of a dense tensor of this shape and type on CUDA device
    `dev`, the current one."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"the current device, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """An output, or a workspace, that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def csa2_norm_rope(xs: Sequence[torch.Tensor], positions, weights=None, outs=None, norms=None,
                   rope_dim=64, eps: float = 1e-6, rope_base: float = 0.0, stream=None) -> list:
    """RMS norm of every head and the rotation of its last rope_dim channels
    by its token's position, for up to 8 tensors in one launch.

    xs: bf16 or fp32 tensors [n, heads, dim] or [n, dim], channels contiguous
    (slices of a wider projection are taken as they are); positions: int64
    [n], or one per tensor (None where nothing is rotated); weights: per tensor
    None or fp32 [dim]; outs: per tensor the output, bf16 or fp32 (None: like
    x; x itself: in place);
    norms: per tensor whether to norm (default: all); rope_dim: one number or
    one per tensor, 0 for no rotation.  Returns the outputs."""
    n = len(xs)
    if n > 8:
        raise ValueError("csa2_norm_rope: at most 8 tensors")
    if outs is None:
        outs = [None] * n
    one_pos = positions is None or isinstance(positions, torch.Tensor)
    one_dim = isinstance(rope_dim, int)
    if (len(outs) != n or (weights is not None and len(weights) != n)
            or (norms is not None and len(norms) != n)
            or (not one_pos and len(positions) != n) or (not one_dim and len(rope_dim) != n)):
        raise ValueError("csa2_norm_rope: one entry per tensor expected")
    outs = [_empty(x.shape, x.dtype, x.device, stream) if y is None else y for x, y in zip(xs, outs)]
    dev = torch.cuda.current_device()
    bf16, f32 = torch.bfloat16, torch.float32
    parts, pos, pos_at, n_pos = [], None, 0, -1
    for i in range(n):
        x, y = xs[i], outs[i]
        shape, xt, yt, sx, sy = x.shape, x.dtype, y.dtype, x.stride(), y.stride()
        if (len(shape) not in (2, 3) or y.shape != shape or x.get_device() != dev
                or y.get_device() != dev or (xt != bf16 and xt != f32)
                or (yt != bf16 and yt != f32)):
            raise ValueError("csa2_norm_rope: bf16 or fp32 tensors [n, heads, dim] or [n, dim] on "
                             "the current device expected")
        if (sx[-1] != 1 or sy[-1] != 1) and shape[-1] > 1:
            raise ValueError("csa2_norm_rope: the channels of a head must be contiguous")
        tokens, dim, r, w = shape[0], shape[-1], rope_dim if one_dim else rope_dim[i], 0
        if r:
            p = positions if one_pos else positions[i]
            if p is not pos or tokens != n_pos:   # once for tensors that share them
                if p is None:
                    raise ValueError("csa2_norm_rope: positions expected where rope_dim is not 0")
                pos, n_pos = p, tokens
                pos_at = _shaped(p, (tokens,), torch.int64, "positions", dev)
        if weights is not None and weights[i] is not None:
            w = _shaped(weights[i], (dim,), f32, "weight", dev)
        if len(shape) == 3:
            heads, xh, yh = shape[1], sx[1], sy[1]
            if heads == 0:
                tokens, heads = 0, 1
        else:
            heads, xh, yh = 1, 0, 0
        parts.append(_NORM_PART.pack(x.data_ptr(), y.data_ptr(), w, pos_at if r else 0, tokens,
                                     sx[0], xh, sy[0], yh, heads, dim, r,
                                     1 if norms is None or norms[i] else 0, xt == f32, yt == f32))
    _check(lib.csa2_norm_rope(n, b"".join(parts), eps, rope_base, _stream(stream, dev)),
           "csa2_norm_rope")
    return outs


# ------------------------------------------------------------------ trees of drafted tokens
class Tree:
    """The trees of drafted tokens of one step (csa2_tree_t), kept on the host.

    parents: per sequence the parent of each draft (an earlier draft of the
    same tree, or -1 for the last committed token); pos0: committed tokens of
    each sequence; seq_ids: the cache's sequences (default: 0, 1, ...).
    Queries are the drafts of all sequences in order."""

    def __init__(self, parents: Sequence[Sequence[int]], pos0: Sequence[int],
                 seq_ids: Optional[Sequence[int]] = None):
        self.n_seqs = len(parents)
        if len(pos0) != self.n_seqs or (seq_ids is not None and len(seq_ids) != self.n_seqs):
            raise ValueError("Tree: one pos0 (and sequence) per tree expected")
        self.n_draft = [len(p) for p in parents]
        self.n_queries = sum(self.n_draft)
        self.pos0 = [int(p) for p in pos0]
        self._n = _i32_array(self.n_draft)
        self._pos0 = _i64_array(pos0)
        self._parent = _i32_array([a for p in parents for a in p])
        self._seq = _i32_array(seq_ids)
        addr = ctypes.addressof
        self.struct = TreeStruct(self.n_seqs, addr(self._seq) if self._seq is not None else None,
                                 addr(self._n), addr(self._pos0), addr(self._parent))
        self.ref = ctypes.byref(self.struct)
        self.depths, self.paths = [], []
        for p in parents:
            d, m = (ctypes.c_int32 * 64)(), (ctypes.c_uint64 * 64)()
            _check(lib.csa2_tree_paths(len(p), _i32_array(p), d, m), "csa2_tree_paths")
            self.depths.append(list(d[:len(p)]))
            self.paths.append(list(m[:len(p)]))

    def positions(self, device=None) -> torch.Tensor:
        """int64 [n_queries]: the drafts' positions (for csa2_norm_rope)."""
        pos = [p + d for p, ds in zip(self.pos0, self.depths) for d in ds]
        return torch.tensor(pos, dtype=torch.int64,
                            device=torch.device("cuda") if device is None else device)

    def owners(self, ratio: int) -> list:
        """Per sequence the drafts that complete a block of `ratio` tokens:
        the ones whose entries are appended before the step, in this order."""
        return [[t for t, d in enumerate(ds) if (p + d + 1) % ratio == 0]
                for p, ds in zip(self.pos0, self.depths)]


def csa2_index_scores_tree(cache: Cache, tree: Tree, q_idx: torch.Tensor, w: torch.Tensor,
                           scores: torch.Tensor, key_hist: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """Index scores of the drafts: q_idx bf16 [n_queries, 32, 128], w fp32
    [n_queries, 32], scores fp32 [n_queries, ld]: the committed entries' scores,
    then those of the draft's path; key_hist: int32 [n_queries, 2048] (bf16
    keys)."""
    nq, c, dev = tree.n_queries, cache.cfg, torch.cuda.current_device()
    ld = scores.shape[-1]
    _check(lib.csa2_index_scores_tree(
        cache.handle, tree.ref,
        _shaped(q_idx, (nq, c.idx_heads, c.idx_dim), torch.bfloat16, "q_idx", dev),
        _shaped(w, (nq, c.idx_heads), torch.float32, "w", dev),
        _shaped(scores, (nq, ld), torch.float32, "scores", dev), ld,
        None if key_hist is None else _shaped(key_hist, (nq, 2048), torch.int32, "key_hist", dev),
        _stream(stream, dev)), "csa2_index_scores_tree")
    return scores


def csa2_index_topk_tree(cache: Cache, tree: Tree, q_idx: torch.Tensor, w: torch.Tensor,
                         topk_idx: Optional[torch.Tensor] = None,
                         topk_score: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Selection of the drafts among the committed entries and their path's;
    int32 [n_queries, topk] entries of the cache, ascending, -1 padded."""
    nq, c, dev = tree.n_queries, cache.cfg, torch.cuda.current_device()
    if topk_idx is None:
        topk_idx = _empty((nq, c.topk), torch.int32, q_idx.device, stream)
    ws = workspace
    if ws is None:
        ws = _empty(max(16, csa2_index_workspace_bytes(cache, nq)), torch.uint8, q_idx.device, stream)
    elif ws.get_device() != dev:
        raise ValueError("workspace: expected on the current device")
    _check(lib.csa2_index_topk_tree(
        cache.handle, tree.ref,
        _shaped(q_idx, (nq, c.idx_heads, c.idx_dim), torch.bfloat16, "q_idx", dev),
        _shaped(w, (nq, c.idx_heads), torch.float32, "w", dev),
        _shaped(topk_idx, (nq, c.topk), torch.int32, "topk_idx", dev),
        None if topk_score is None else _shaped(topk_score, (nq, c.topk), torch.float32,
                                                "topk_score", dev),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream, dev)), "csa2_index_topk_tree")
    return topk_idx


def csa2_sparse_attn_tree(cache: Cache, tree: Tree, q: torch.Tensor,
                          swa_kv: Optional[torch.Tensor], draft_kv: Optional[torch.Tensor],
                          topk_idx: torch.Tensor, scale: float,
                          swa_len: Optional[Sequence[int]] = None,
                          out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None,
                          sink: Optional[torch.Tensor] = None, rope_out: bool = False,
                          rope_base: float = 0.0, swa_fp8=None, draft_fp8=None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Readout of the drafts of one layer; see csa2_sparse_attn_tree_layers."""
    return csa2_sparse_attn_tree_layers(
        cache, tree, [q], None if swa_kv is None else [swa_kv],
        None if draft_kv is None else [draft_kv], topk_idx, scale,
        None if out is None else [out], lses=None if lse is None else [lse], swa_len=swa_len,
        sinks=None if sink is None else [sink], rope_out=rope_out, rope_base=rope_base,
        swa_fp8s=None if swa_fp8 is None else [swa_fp8],
        draft_fp8s=None if draft_fp8 is None else [draft_fp8], workspace=workspace,
        stream=stream)[0]


def csa2_sparse_attn_tree_layers(cache: Cache, tree: Tree, qs: Sequence[torch.Tensor],
                                 swa_kvs: Optional[Sequence[torch.Tensor]],
                                 draft_kvs: Optional[Sequence[torch.Tensor]],
                                 topk_idx: torch.Tensor, scale: float,
                                 outs: Optional[Sequence[torch.Tensor]] = None,
                                 lses: Optional[Sequence[Optional[torch.Tensor]]] = None,
                                 swa_len: Optional[Sequence[int]] = None,
                                 sinks: Optional[Sequence[Optional[torch.Tensor]]] = None,
                                 rope_out: bool = False, rope_base: float = 0.0,
                                 swa_fp8s=None, draft_fp8s=None,
                                 workspace: Optional[torch.Tensor] = None, stream=None) -> list:
    """Readout of the drafts for several layers of a group in one launch.

    Per layer: q bf16 [n_queries, heads, 512]; committed window rows swa_kv
    bf16 [n_seqs, swa, 512] (the first swa_len[i] rows are the newest
    committed rows, in position order) and the drafts' rows draft_kv bf16
    [n_queries, 512], or both as the triples of csa2_swa_fp8_quantise;
    swa_len: host, default min(swa, pos0); topk_idx from
    csa2_index_topk_tree; rope_out rotates each output by minus its draft's
    position.  workspace as for csa2_sparse_attn_decode.  Returns the
    outputs."""
    nq, S, c, L = tree.n_queries, tree.n_seqs, cache.cfg, len(qs)
    H, D, W, bf16 = c.n_heads, c.head_dim, c.swa, torch.bfloat16
    dev = torch.cuda.current_device()
    if outs is None:
        outs = [_empty(q.shape, q.dtype, q.device, stream) for q in qs]
    for xs in (outs, lses, sinks, swa_kvs, draft_kvs, swa_fp8s, draft_fp8s):
        if xs is not None and len(xs) != L:
            raise ValueError("csa2_sparse_attn_tree_layers: one entry per layer expected")
    if (swa_fp8s is None) != (draft_fp8s is None):
        raise ValueError("csa2_sparse_attn_tree_layers: window and drafted rows of one format")
    if swa_len is not None and len(swa_len) != S:
        raise ValueError("csa2_sparse_attn_tree_layers: one swa_len per tree expected")
    if W and swa_fp8s is None and (swa_kvs is None or draft_kvs is None):
        raise ValueError("csa2_sparse_attn_tree_layers: window and drafted rows expected")

    def fp8(rows, n, what):
        codes, rope, scales = rows
        return (_shaped(codes.view(n, codes.shape[-1]), (n, 448), torch.uint8, what, dev),
                _shaped(rope.view(n, rope.shape[-1]), (n, 64), bf16, what, dev),
                _shaped(scales.view(n, scales.shape[-1]), (n, 8), torch.uint8, what, dev))

    layers = []
    for l in range(L):
        lse = None if lses is None else lses[l]
        sink = None if sinks is None else sinks[l]
        swa = draft = 0
        f8 = (0, 0, 0, 0, 0, 0)
        if W and swa_fp8s is not None:
            f8 = fp8(swa_fp8s[l], S * W, "swa_fp8") + fp8(draft_fp8s[l], nq, "draft_fp8")
        elif W:
            swa = _shaped(swa_kvs[l], (S, W, D), bf16, "swa_kv", dev)
            draft = _shaped(draft_kvs[l], (nq, D), bf16, "draft_kv", dev)
        layers.append(_TREE_LAYER.pack(
            _shaped(qs[l], (nq, H, D), bf16, "q", dev), swa, draft,
            _shaped(outs[l], (nq, H, D), bf16, "out", dev),
            0 if lse is None else _shaped(lse, (nq, H), torch.float32, "lse", dev),
            0 if sink is None else _shaped(sink, (H,), torch.float32, "sink", dev), *f8))
    ws, nbytes = (cache._token, 16) if workspace is None else (
        workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(lib.csa2_sparse_attn_tree(
        cache.handle, tree.ref, L, b"".join(layers), _i32_array(swa_len),
        _shaped(topk_idx, (nq, c.topk), torch.int32, "topk_idx", dev), scale, 1 if rope_out else 0,
        rope_base, ws if nbytes else None, nbytes, _stream(stream, dev)), "csa2_sparse_attn_tree")
    return list(outs)


def csa2_cache_accept_tree(cache: Cache, tree: Tree, accepted: Sequence[int], stream=None):
    """Commits, per sequence, the path of draft accepted[i] (-1: none): its
    entries stay, the other drafts' are dropped."""
    if len(accepted) != tree.n_seqs:
        raise ValueError("csa2_cache_accept_tree: one accepted draft (or -1) per tree expected")
    _check(lib.csa2_cache_accept_tree(cache.handle, tree.ref, _i32_array(accepted),
                                      _stream(stream)), "csa2_cache_accept_tree")


# ------------------------------------------------------------------ window rows in a cache
class Window:
    """The newest `swa` rows of every sequence of one layer, and those of its
    first n_first tokens, in torch-owned memory (csa2_window_t): in 8 bits, or
    as bf16 (fp8=False).  `swa_kv` and `swa_fp8` are the rows as
    csa2_sparse_attn_decode takes them, without a copy."""

    def __init__(self, n_seqs: int, swa: int = 128, n_first: int = 0, fp8: bool = True, device=None,
                 stream=None):
        if n_seqs < 0 or not 1 <= swa <= 128 or not 0 <= n_first <= 8:
            raise ValueError("Window: n_seqs of at least 0, swa of 1 to 128 and n_first of 0 to 8 "
                             "expected")
        self.n_seqs, self.swa, self.n_first, self.fp8 = n_seqs, swa, n_first, bool(fp8)
        device = torch.device("cuda") if device is None else torch.device(device)
        n = max(1, n_seqs * (swa + n_first))

        def empty(shape, dtype):
            return _empty(shape, dtype, device, stream)

        self.rows = self.codes = self.rope = self.scales = None
        if self.fp8:
            self.codes, self.rope = empty((n, 448), torch.uint8), empty((n, 64), torch.bfloat16)
            self.scales = empty((n, 8), torch.uint8)
        else:
            self.rows = empty((n, 512), torch.bfloat16)
        self.pos = empty((n,), torch.int64)
        self.error = empty((4,), torch.int32)
        self.device = self.pos.get_device()
        self.waits = (0, 0)    # csa2_window_opts_t: wait_cycles, withhold

        def at(t):
            return None if t is None else t.data_ptr()

        self.struct = WindowStruct(n_seqs, swa, n_first, int(self.fp8), at(self.rows),
                                   at(self.codes), at(self.rope), at(self.scales), at(self.pos),
                                   at(self.error))
        self.ref = ctypes.byref(self.struct)
        self.reset(stream=stream)

    def _here(self, what: str) -> int:
        """The current device, which has to be the cache's."""
        dev = torch.cuda.current_device()
        if dev != self.device:
            raise ValueError(f"{what}: the cache is on device {self.device}, the current one is {dev}")
        return dev

    def reset(self, seq: Optional[int] = None, stream=None):
        """Forgets the rows of sequence seq (None: of all)."""
        dev = self._here("csa2_window_reset")
        _check(lib.csa2_window_reset(self.ref, -1 if seq is None else seq, _stream(stream, dev)),
               "csa2_window_reset")

    def set_wait_limit(self, cycles: int):
        """Bound, in SM clock cycles, on every wait inside the attention kernels
        that read this cache (0: the default); see csa2_window_opts_t."""
        if cycles < 0:
            raise ValueError("Window.set_wait_limit: 0 cycles or more expected")
        self.waits = (cycles, self.waits[1])

    def inject_fault(self, withhold: int):
        """For tests: the queries of the withhold-th item that a CTA works on, and of
        the ones behind it, are not loaded (0: all are); see csa2_window_opts_t."""
        if withhold < 0:
            raise ValueError("Window.inject_fault: 0 or more expected")
        self.waits = (self.waits[0], withhold)

    @property
    def swa_kv(self) -> Optional[torch.Tensor]:
        """bf16 [n_seqs, swa, 512], the window rows (None in 8 bits)."""
        if self.fp8:
            return None
        return self.rows[:self.n_seqs * self.swa].view(self.n_seqs, self.swa, 512)

    @property
    def swa_fp8(self):
        """The window rows in 8 bits (codes, rope, scales); None as bf16."""
        if not self.fp8:
            return None
        n = self.n_seqs * self.swa
        return self.codes[:n], self.rope[:n], self.scales[:n]

    def device_error(self, stream=None) -> int:
        st = ctypes.c_int32()
        dev = self._here("csa2_window_device_error")
        _check(lib.csa2_window_device_error(self.ref, _stream(stream, dev), ctypes.byref(st)),
               "csa2_window_device_error")
        return st.value


def _one_each(what: str, n: int, *lists):
    for xs in lists:
        if xs is not None and len(xs) != n:
            raise ValueError(f"{what}: one entry per segment expected")


def csa2_window_append(win: Window, rows: torch.Tensor, pos: torch.Tensor,
                       n_rows: Optional[Sequence[int]] = None,
                       seq_ids: Optional[Sequence[int]] = None,
                       rounded: Optional[torch.Tensor] = None, stream=None):
    """Writes rows at the end of sequences: rows bf16 [sum n_rows, 512], n_rows[i]
    of them (default: one) for sequence seq_ids[i] (default: i, each at most
    once) at positions pos[i], pos[i] + 1, ...; pos: int64 [segments], negative:
    not stored.  rounded: bf16 like rows, the rows as the cache holds them."""
    dev, n = win._here("csa2_window_append"), pos.numel()
    _one_each("csa2_window_append", n, n_rows, seq_ids)
    total = n if n_rows is None else sum(n_rows)
    _check(lib.csa2_window_append(
        win.ref, n, _i32_array(seq_ids), _i32_array(n_rows),
        _shaped(pos, (n,), torch.int64, "pos", dev),
        _shaped(rows, (total, 512), torch.bfloat16, "rows", dev),
        None if rounded is None else _shaped(rounded, (total, 512), torch.bfloat16, "rounded", dev),
        _stream(stream, dev)), "csa2_window_append")


def csa2_window_read(win: Window, end: torch.Tensor, n_rows: Optional[int] = None,
                     seq_ids: Optional[Sequence[int]] = None, out: Optional[torch.Tensor] = None,
                     first: Optional[torch.Tensor] = None, fp8: bool = False, stream=None):
    """The windows in position order, bf16 [segments, n_rows, 512]: row j of
    segment i is that of position max(0, end[i] - n_rows) + j, zero where it is
    not held or not below end[i].  end: int64 [segments]; n_rows: default swa;
    first: bf16 [segments, n_first, 512], filled with the first tokens' rows;
    fp8: the rows as they are held in 8 bits (codes, rope, scales) instead (out:
    such a triple)."""
    dev, n = win._here("csa2_window_read"), end.numel()
    _one_each("csa2_window_read", n, seq_ids)
    w = win.swa if n_rows is None else n_rows
    where = end.device
    o = [None] * 4
    if fp8:
        if out is None:
            out = (_empty((n * w, 448), torch.uint8, where, stream),
                   _empty((n * w, 64), torch.bfloat16, where, stream),
                   _empty((n * w, 8), torch.uint8, where, stream))
        o[1:] = [_shaped(t, (n * w, d), ty, "out", dev) for t, d, ty in
                 zip(out, (448, 64, 8), (torch.uint8, torch.bfloat16, torch.uint8))]
    else:
        if out is None:
            out = _empty((n, w, 512), torch.bfloat16, where, stream)
        o[0] = _shaped(out, (n, w, 512), torch.bfloat16, "out", dev)
    _check(lib.csa2_window_read(
        win.ref, n, _i32_array(seq_ids), _shaped(end, (n,), torch.int64, "end", dev), w, *o,
        None if first is None else _shaped(first, (n, win.n_first, 512), torch.bfloat16, "first",
                                           dev),
        _stream(stream, dev)), "csa2_window_read")
    return out


def _window_opts(what, nq, heads, lse, sink, rope_out, rope_base, dev, error=None, waits=(0, 0)):
    if lse is None and sink is None and not rope_out and error is None and waits == (0, 0):
        return None
    return ctypes.byref(WindowOpts(
        None if sink is None else _shaped(sink, (heads,), torch.float32, "sink", dev),
        None if lse is None else _shaped(lse, (nq, heads), torch.float32, "lse", dev),
        1 if rope_out else 0, float(rope_base),
        None if error is None else _shaped(error, error.shape, torch.int32, "error", dev), *waits))


def _window_queries(what: str, q: torch.Tensor, nq: int, out, stream, dev: int):
    """(output, pointers of q and output)"""
    if q.dim() != 3 or q.shape[1] not in (64, 128):
        raise ValueError(f"{what}: q of shape [n_queries, 64 or 128, 512] expected")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    shape = (nq, q.shape[1], 512)
    return out, _shaped(q, shape, torch.bfloat16, "q", dev), _shaped(out, shape, torch.bfloat16,
                                                                     "out", dev)


def _draft_rows(win: Window, draft_kv, nq: int, dev: int):
    """Pointers of drafts' rows in the cache's form: bf16, or a triple."""
    if not win.fp8:
        return _shaped(draft_kv, (nq, 512), torch.bfloat16, "draft_kv", dev), None, None, None
    if not isinstance(draft_kv, (tuple, list)) or len(draft_kv) != 3:
        raise ValueError("draft_kv: the triple of csa2_swa_fp8_quantise expected, as the cache is in "
                         "8 bits")
    return (None, *[_shaped(t, (nq, d), ty, "draft_kv", dev) for t, d, ty in
                    zip(draft_kv, (448, 64, 8), (torch.uint8, torch.bfloat16, torch.uint8))])


def csa2_window_attn_decode(win: Window, q: torch.Tensor, pos: torch.Tensor, scale: float,
                            seq_ids: Optional[Sequence[int]] = None,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            sink: Optional[torch.Tensor] = None, rope_out: bool = False,
                            rope_base: float = 0.0, stream=None) -> torch.Tensor:
    """Attention of a window layer, one token a sequence: q bf16 [n_queries, 64
    or 128, 512] at positions pos (int64 [n_queries]; negative: sees nothing)
    of sequences seq_ids (default: 0, 1, ...) over the rows that the cache
    holds, the query's own among them (csa2_window_append comes first).  lse,
    sink and rope_out as for csa2_sparse_attn_decode."""
    dev, nq = win._here("csa2_window_attn_decode"), q.shape[0]
    _one_each("csa2_window_attn_decode", nq, seq_ids)
    out, q_at, out_at = _window_queries("csa2_window_attn_decode", q, nq, out, stream, dev)
    _check(lib.csa2_window_attn_decode(
        win.ref, q.shape[1], nq, _i32_array(seq_ids), q_at,
        _shaped(pos, (nq,), torch.int64, "pos", dev), scale, out_at,
        _window_opts("csa2_window_attn_decode", nq, q.shape[1], lse, sink, rope_out, rope_base, dev,
                     waits=win.waits),
        _stream(stream, dev)), "csa2_window_attn_decode")
    return out


def csa2_window_attn_tree(win: Window, tree: Tree, q: torch.Tensor, draft_kv, scale: float,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          sink: Optional[torch.Tensor] = None, rope_out: bool = False,
                          rope_base: float = 0.0, stream=None) -> torch.Tensor:
    """The same for the drafts of a tree: q bf16 [n_queries, heads, 512];
    draft_kv: the drafts' rows in the cache's form, bf16 [n_queries, 512] or
    the triple of csa2_swa_fp8_quantise."""
    dev, nq = win._here("csa2_window_attn_tree"), tree.n_queries
    out, q_at, out_at = _window_queries("csa2_window_attn_tree", q, nq, out, stream, dev)
    _check(lib.csa2_window_attn_tree(
        win.ref, tree.ref, q.shape[1], q_at, *_draft_rows(win, draft_kv, nq, dev), scale, out_at,
        _window_opts("csa2_window_attn_tree", nq, q.shape[1], lse, sink, rope_out, rope_base, dev,
                     waits=win.waits),
        _stream(stream, dev)), "csa2_window_attn_tree")
    return out


def csa2_window_accept_tree(win: Window, tree: Tree, draft_kv, accepted: torch.Tensor, stream=None):
    """Writes the rows of each tree's accepted path (accepted: int32 [n_seqs]
    on the device, as csa2_verify_tree gives it; -1: none)."""
    dev = win._here("csa2_window_accept_tree")
    _check(lib.csa2_window_accept_tree(
        win.ref, tree.ref, _shaped(accepted, (tree.n_seqs,), torch.int32, "accepted", dev),
        *_draft_rows(win, draft_kv, tree.n_queries, dev), _stream(stream, dev)),
        "csa2_window_accept_tree")


def csa2_window_attn_prefill(q: torch.Tensor, pos0: int, rows: torch.Tensor, rows_pos0: int,
                             scale: float, swa: int = 128, n_first: int = 0,
                             first: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None,
                             sink: Optional[torch.Tensor] = None, rope_out: bool = False,
                             rope_base: float = 0.0, error: Optional[torch.Tensor] = None,
                             wait_cycles: int = 0, withhold: int = 0,
                             stream=None) -> torch.Tensor:
    """The same for a chunk of one sequence: query i at position pos0 + i; row r
    of rows (bf16 [n, 512]) is that of position rows_pos0 + r, the chunk's rows
    and those before it (csa2_window_read); first: bf16 [n_first, 512], the
    first tokens' rows where rows_pos0 is not 0; error: int32, the sticky error
    word of the call (Window.error); wait_cycles, withhold: as Window.set_wait_limit
    and Window.inject_fault set them."""
    what, dev, nq = "csa2_window_attn_prefill", torch.cuda.current_device(), q.shape[0]
    out, q_at, out_at = _window_queries(what, q, nq, out, stream, dev)
    n = rows.shape[0]
    _check(lib.csa2_window_attn_prefill(
        q.shape[1], nq, pos0, q_at, _shaped(rows, (n, 512), torch.bfloat16, "rows", dev), rows_pos0,
        n, swa, None if first is None else _shaped(first, (n_first, 512), torch.bfloat16, "first", dev),
        n_first, scale, out_at,
        _window_opts(what, nq, q.shape[1], lse, sink, rope_out, rope_base, dev, error,
                     (wait_cycles, withhold)),
        _stream(stream, dev)), what)
    return out


# ------------------------------------------------------------------ verification of drafts
def _value_rows(t: torch.Tensor, n: int, vocab: int, dtype, what: str, dev: int):
    """Device pointer and row distance of [n, vocab] values on CUDA device `dev`,
    a row's next to each other."""
    step, one = t.stride() if t.dim() == 2 else (0, 0)
    if t.shape != (n, vocab) or t.dtype != dtype or t.get_device() != dev or (one != 1 and vocab > 1):
        raise ValueError(f"{what}: expected {dtype} [{n}, {vocab}] on the current device, with the "
                         f"values of a row next to each other")
    return t.data_ptr(), step


def csa2_verify_tree(tree: Tree, tokens: torch.Tensor, logits: torch.Tensor,
                     temperature: Optional[torch.Tensor] = None,
                     uniform: Optional[torch.Tensor] = None, noise: Optional[torch.Tensor] = None,
                     root_logits: Optional[torch.Tensor] = None,
                     draft_logits: Optional[torch.Tensor] = None,
                     draft_root: Optional[torch.Tensor] = None,
                     accepted: Optional[torch.Tensor] = None,
                     next_token: Optional[torch.Tensor] = None, stream=None):
    """Which drafts are kept, by rejection sampling against the target's
    probabilities, and the token that follows them: (accepted, next_token),
    int32 [n_seqs] on the device; accepted is the last accepted draft of each
    tree (-1: none), as csa2_window_accept_tree takes it (csa2_cache_accept_tree
    wants it on the host).

    tokens: int32 [n_queries], the drafts'; logits: bf16 or fp32 [n_queries,
    vocab], the target's after each draft, root_logits [n_seqs, vocab] those
    after the last committed token (None: the first draft of each tree is the
    token that the step before has drawn, and is kept); draft_logits and
    draft_root: likewise those of the model that drafted (None: drafts count as
    certain); temperature: fp32 [n_seqs] (None: 0), 0 (or below 2^-100) takes the
    largest logit;
    uniform: fp32 [n_queries] in [0, 1); noise: fp32 [n_seqs, vocab],
    exponential variates.  Rows may be further apart than vocab (the same for
    all logits); rows at 16-byte boundaries are read faster.

    draft_logits are for children that were drawn from softmax(draft /
    temperature) independently of each other, in call order; others (the most
    likely ones, or drawn without replacement) are verified without, or the tokens
    are not distributed as the target's."""
    what, dev, nq, S = "csa2_verify_tree", torch.cuda.current_device(), tree.n_queries, tree.n_seqs
    if logits.dim() != 2 or logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{what}: logits bf16 or fp32 [n_queries, vocab] expected")
    vocab, dtype = logits.shape[1], logits.dtype
    f32, i32 = torch.float32, torch.int32
    ld, at = None, []
    for t, n, name in ((logits, nq, "logits"), (root_logits, S, "root_logits"),
                       (draft_logits, nq, "draft_logits"), (draft_root, S, "draft_root")):
        if t is None:
            at.append(None)
            continue
        p, step = _value_rows(t, n, vocab, dtype, name, dev)
        if n > 1:   # a single row has no distance to the next
            if ld is not None and step != ld:
                raise ValueError(f"{name}: the rows of all logits have to be equally far apart")
            ld = step
        at.append(p)
    noise_at, noise_ld = None, 0
    if noise is not None:
        noise_at, noise_ld = _value_rows(noise, S, vocab, f32, "noise", dev)
        if S == 1:
            noise_ld = (vocab + 3) // 4 * 4
    if accepted is None:
        accepted = _empty((S,), i32, logits.device, stream)
    if next_token is None:
        next_token = _empty((S,), i32, logits.device, stream)
    v = VerifyStruct(
        vocab, dtype is f32, _shaped(tokens, (nq,), i32, "tokens", dev), *at,
        (vocab + 7) // 8 * 8 if ld is None else ld,
        None if temperature is None else _shaped(temperature, (S,), f32, "temperature", dev),
        None if uniform is None else _shaped(uniform, (nq,), f32, "uniform", dev),
        noise_at, noise_ld, _shaped(accepted, (S,), i32, "accepted", dev),
        _shaped(next_token, (S,), i32, "next_token", dev))
    _check(lib.csa2_verify_tree(tree.ref, ctypes.byref(v), _stream(stream, dev)), what)
    return accepted, next_token
