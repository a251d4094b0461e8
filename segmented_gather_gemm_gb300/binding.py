"""ctypes binding of libcsgmv.so (include/csgmv.h), same names as the C ABI.

Argument marshalling only: torch supplies device memory and the current CUDA
stream, every step of the path runs in the library's kernels.  There is no
fallback: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsgmv.so")

CSGMV_DTYPE_BF16 = 0
CSGMV_DTYPE_F32 = 1
CSGMV_DTYPE_F16 = 2

STATUS_BITS = {
    1: "BAD_ADAPTER", 2: "BAD_RANK", 4: "BAD_TOKEN_ID", 8: "BAD_PERMUTATION", 16: "CAPACITY", 32: "BAD_LENS",
}

# bits of KvCache.status and DraftTree.status (CSGMV_KV_STATUS_*; 1 << 30: a
# bounded wait inside a kernel ran out)
KV_STATUS_BITS = {
    1: "BAD_SEQ", 2: "BAD_PAGE", 4: "CAPACITY", 8: "BAD_LENS", 16: "BAD_TREE", 32: "BAD_TOKEN",
    64: "BAD_VALUE", 1 << 30: "TIMEOUT",
}

EXPORTED = ["csgmv_last_error", "csgmv_version", "csgmv_chunk_size", "csgmv_batch_info_capacity",
            "csgmv_build_batch_info", "csgmv_build_lm_head_batch_info", "csgmv_shrink", "csgmv_expand", "csgmv_qkv", "csgmv_qkv_workspace_bytes",
            "csgmv_qkv_static_scratch", "embedding_lora_a", "embedding_lora_a_extra", "extra_token_embedding",
            "csgmv_expand_sliced", "csgmv_qkv_sliced", "csgmv_qkv_path", "csgmv_tile_table_ints",
            "embedding_lora_a_transposed", "csgmv_transpose_embedding",
            "csgmv_kv_scratch_ints", "csgmv_kv_commit", "csgmv_kv_fork", "csgmv_kv_free", "csgmv_kv_compact",
            "csgmv_kv_copy_pages", "csgmv_tree_attention", "csgmv_tree_attention_workspace_bytes",
            "csgmv_build_draft_tree", "csgmv_verify_drafts", "csgmv_add_norm", "csgmv_rope_turns",
            "csgmv_rotary", "csgmv_kv_extend", "csgmv_kv_append", "csgmv_count_tokens", "csgmv_count_reset",
            "csgmv_count_fork", "csgmv_process_logits"]

# csgmv_qkv_path results (CSGMV_PATH_*)
PATHS = {0: "fused", 1: "decode", 2: "small_split", 3: "stream"}


class CsgmvError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"csgmv error {code}: {msg}")
        self.code = code


class _BatchInfoC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "seg_indptr", "weight_indices", "permutation", "lora_ranks", "scalings", "num_segments_dev",
        "max_len_dev", "req_seg_indptr", "req_weight_indices", "status")] + [
        (n, ctypes.c_int32) for n in (
            "max_segments", "max_tokens", "max_loras", "max_bs", "max_rank",
            "num_tokens", "chunk_size", "bs", "num_loras", "use_cuda_graph")] + [
        ("tile_table", ctypes.c_void_p)]


class _KvCacheC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k_pages", "v_pages", "page_table", "seq_lens", "page_refs", "scratch", "status")] + [
        (n, ctypes.c_int64) for n in ("layer_stride", "page_stride", "head_stride", "token_stride")] + [
        (n, ctypes.c_int32) for n in (
            "dtype", "num_layers", "num_pages", "page_size", "num_kv_heads", "head_dim", "max_seqs",
            "max_pages_per_seq")]


class _NormC(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("eps", ctypes.c_float), ("kind", ctypes.c_int32)]


class _RopeC(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("scale", ctypes.c_float), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class _TokenCountsC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("counts", "seen", "num_seen", "status")] + [
        ("max_seqs", ctypes.c_int32), ("vocab_size", ctypes.c_int32)]


class _LogitRulesC(ctypes.Structure):
    _fields_ = [("counts", ctypes.POINTER(_TokenCountsC))] + [(n, ctypes.c_void_p) for n in (
        "repetition", "frequency", "presence", "temperature", "bias_indptr", "bias_tokens", "bias_values", "allow",
        "allow_index")] + [("bias_total", ctypes.c_int64), ("num_allow", ctypes.c_int32), ("allow_words", ctypes.c_int32),
                           ("status", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded libcsgmv.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with segmented_gather_gemm_gb300.build "
                           "(the csgmv path has no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    i32p = ctypes.POINTER(ctypes.c_int32)
    bip = ctypes.POINTER(_BatchInfoC)
    kvp = ctypes.POINTER(_KvCacheC)
    f32, size_t = ctypes.c_float, ctypes.c_size_t
    sig = {
        "csgmv_last_error": (ctypes.c_char_p, []),
        "csgmv_version": (ctypes.c_char_p, []),
        "csgmv_chunk_size": (i32, [i32, i32]),
        "csgmv_batch_info_capacity": (i32, [i32, i32, i32p, i32p]),
        "csgmv_build_batch_info": (i32, [bip, vp, vp, i32, i32, vp, vp, i32, i32, i32, i32, vp]),
        "csgmv_build_lm_head_batch_info": (i32, [bip, vp, vp, i32, i32, vp, vp, i32, i32, i32, i32, vp]),
        "csgmv_shrink": (i32, [vp, i64, i64, vp, i32, vp, i32, i64, bip, vp]),
        "csgmv_expand": (i32, [vp, i32, i64, vp, i64, i32p, i32, i32, vp, i32, bip, vp]),
        "csgmv_qkv": (i32, [vp, i64, vp, vp, i64, i32p, i32, i32, vp, vp, ctypes.c_size_t, bip, vp]),
        "csgmv_qkv_workspace_bytes": (ctypes.c_size_t, [bip, i32]),
        "csgmv_qkv_static_scratch": (i32, [vp, i64, vp, vp, i64, i32p, i32, i32, vp, bip, vp]),
        "embedding_lora_a": (i32, [vp, vp, i64, i32, vp, bip, vp]),
        "embedding_lora_a_extra": (i32, [vp, vp, i64, i32, vp, i64, vp, bip, vp]),
        "csgmv_expand_sliced": (i32, [vp, i32, i64, ctypes.POINTER(vp), i64, i32p, i32, i32, vp, i32, bip, vp]),
        "csgmv_qkv_sliced": (i32, [vp, i64, vp, ctypes.POINTER(vp), i64, i32p, i32, i32, vp, vp, ctypes.c_size_t,
                                   bip, vp]),
        "extra_token_embedding": (i32, [vp, vp, i64, vp, i64, i64, bip, vp]),
        "csgmv_qkv_path": (i32, [bip, i64, i64, i32p, i32, ctypes.c_size_t]),
        "csgmv_tile_table_ints": (i64, [i32, i32]),
        "embedding_lora_a_transposed": (i32, [vp, vp, i64, i32, vp, i64, vp, bip, vp]),
        "csgmv_transpose_embedding": (i32, [vp, i64, i32, i64, vp, vp]),
        "csgmv_kv_scratch_ints": (i64, [i32, i32]),
        "csgmv_kv_commit": (i32, [kvp, vp, vp, i64, i64, i64, i64, vp, i32, vp, vp, vp, i32, vp]),
        "csgmv_kv_fork": (i32, [kvp, vp, vp, i32, vp]),
        "csgmv_kv_free": (i32, [kvp, vp, vp, i32, vp]),
        "csgmv_kv_compact": (i32, [kvp, vp]),
        "csgmv_kv_copy_pages": (i32, [kvp, vp, vp, i32, vp]),
        "csgmv_tree_attention": (i32, [vp, i64, i64, i32, vp, vp, i64, i64, kvp, i32, vp, vp, i32, i64, vp, i32, f32,
                                       vp, i64, i64, vp, vp, size_t, vp]),
        "csgmv_tree_attention_workspace_bytes": (size_t, [kvp, i32]),
        "csgmv_build_draft_tree": (i32, [vp, vp, i32, i64, i32, vp, vp, vp, vp, vp, vp]),
        "csgmv_verify_drafts": (i32, [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, i32, i64, i32, vp, i32, vp, vp, vp,
                                      vp]),
        "csgmv_add_norm": (i32, [vp, i64, i32, vp, i64, i32, vp, i64, ctypes.POINTER(_NormC), ctypes.POINTER(_NormC), f32,
                                 i64, i32, vp, i64, vp, i64, vp]),
        "csgmv_rope_turns": (i32, [vp, i32, vp]),
        "csgmv_rotary": (i32, [ctypes.POINTER(_RopeC), i32, i32, vp, i64, vp, i64, i64, i32, vp, i64, i64, i32, vp, i64, i64,
                               vp, i64, i64, i32, vp]),
        "csgmv_kv_extend": (i32, [kvp, vp, vp, vp, i32, i64, vp, vp, vp, vp]),
        "csgmv_kv_append": (i32, [kvp, i32, ctypes.POINTER(_RopeC), vp, vp, i64, vp, i64, i64, i32, vp, i64, i64, vp, i64, i64,
                                  vp, i64, i64, vp, i64, i64, vp]),
        "csgmv_count_tokens": (i32, [ctypes.POINTER(_TokenCountsC), vp, i64, vp, vp, i32, vp, vp, i32, i32, vp]),
        "csgmv_count_reset": (i32, [ctypes.POINTER(_TokenCountsC), vp, i32, vp]),
        "csgmv_count_fork": (i32, [ctypes.POINTER(_TokenCountsC), vp, vp, i32, vp]),
        "csgmv_process_logits": (i32, [vp, i32, i64, vp, vp, i32, i64, i32, ctypes.POINTER(_LogitRulesC), vp, vp, i32, i32, vp,
                                       i64, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def _check(rc: int):
    if rc != 0:
        raise CsgmvError(rc, lib().csgmv_last_error().decode())


def _stream(stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor | None):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _offsets(offsets) -> ctypes.Array:
    vals = [int(v) for v in (offsets.tolist() if hasattr(offsets, "tolist") else offsets)]
    return (ctypes.c_int32 * len(vals))(*vals)


def csgmv_version() -> str:
    return lib().csgmv_version().decode()


def csgmv_chunk_size(num_tokens: int, max_chunk_size: int) -> int:
    return int(lib().csgmv_chunk_size(int(num_tokens), int(max_chunk_size)))


def csgmv_batch_info_capacity(max_bs: int, num_tokens_per_bs: int) -> tuple[int, int]:
    ms, mt = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib().csgmv_batch_info_capacity(int(max_bs), int(num_tokens_per_bs), ctypes.byref(ms),
                                           ctypes.byref(mt)))
    return int(ms.value), int(mt.value)


def tile_table_ints(max_loras: int, max_tokens: int) -> int:
    """int32 entries of a batch info's tile table (csgmv_tile_table_ints)."""
    return 4 * (max(max_loras, 0) + max(max_tokens, 0) // 64 + 2)


def csgmv_tile_table_ints(max_loras: int, max_tokens: int) -> int:
    return int(lib().csgmv_tile_table_ints(int(max_loras), int(max_tokens)))


class BatchInfo:
    """Device buffers of one batch info (caller-owned, allocated once by torch)
    plus the C struct that points at them."""

    def __init__(self, max_bs: int, max_tokens: int, max_segments: int, max_loras: int, max_rank: int,
                 device="cuda", with_request_fields: bool = True, with_tile_table: bool = True):
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.seg_indptr = torch.zeros(max_segments + 1, **i32)
        self.weight_indices = torch.zeros(max(max_segments, 1), **i32)
        self.permutation = torch.zeros(max(max_tokens, 1), **i32)
        self.lora_ranks = torch.zeros(max_loras, **i32)
        self.scalings = torch.zeros(max_loras, dtype=torch.float32, device=dev)
        self.num_segments = torch.zeros(1, **i32)
        self.max_len = torch.zeros(1, **i32)
        self.status = torch.zeros(1, **i32)
        self.req_seg_indptr = torch.zeros(max_bs + 1, **i32) if with_request_fields else None
        self.req_weight_indices = torch.zeros(max(max_bs, 1), **i32) if with_request_fields else None
        self.tile_table = torch.zeros(tile_table_ints(max_loras, max_tokens), **i32) if with_tile_table else None
        c = _BatchInfoC()
        for n in ("seg_indptr", "weight_indices", "permutation", "lora_ranks", "scalings", "status",
                  "req_seg_indptr", "req_weight_indices", "tile_table"):
            t = getattr(self, n)
            setattr(c, n, t.data_ptr() if t is not None else None)
        c.num_segments_dev = self.num_segments.data_ptr()
        c.max_len_dev = self.max_len.data_ptr()
        c.max_segments, c.max_tokens, c.max_loras = max_segments, max_tokens, max_loras
        c.max_bs, c.max_rank = max_bs, max_rank
        c.num_tokens = -1
        self.c = c

    @classmethod
    def for_cuda_graph(cls, max_bs: int, num_tokens_per_bs: int, max_loras: int, max_rank: int, **kw):
        """Capacities of chunked_backend.py init_cuda_graph_batch_info."""
        ms, mt = csgmv_batch_info_capacity(max_bs, num_tokens_per_bs)
        return cls(max_bs, mt, ms, max_loras, max_rank, **kw)

    @classmethod
    def for_batch(cls, bs: int, num_tokens: int, max_loras: int, max_rank: int, min_chunk: int = 16, **kw):
        """Capacities that fit one eager batch of bs requests and num_tokens
        tokens at any chunk size >= min_chunk: ceil(s / min_chunk) full
        segments plus one partial segment per slot run."""
        ms = (num_tokens + min_chunk - 1) // min_chunk + min(max(bs, 1), max_loras)
        return cls(max(bs, 1), num_tokens, ms, max_loras, max_rank, **kw)

    @property
    def num_tokens(self) -> int:
        return int(self.c.num_tokens)

    @property
    def chunk_size(self) -> int:
        return int(self.c.chunk_size)

    def device_status(self) -> int:
        return int(self.status.item())


def csgmv_build_batch_info(bi: BatchInfo, req_lens: torch.Tensor, req_adapter: torch.Tensor, num_tokens: int,
                           lora_ranks: torch.Tensor, scalings: torch.Tensor, max_chunk_size: int = 128,
                           chunk_size_override: int = 0, use_cuda_graph: bool = False, stream=None) -> None:
    bs = int(req_lens.numel())
    _check(lib().csgmv_build_batch_info(ctypes.byref(bi.c), _ptr(req_lens), _ptr(req_adapter), bs,
                                        int(num_tokens), _ptr(lora_ranks), _ptr(scalings),
                                        int(lora_ranks.numel()), int(max_chunk_size),
                                        int(chunk_size_override), int(bool(use_cuda_graph)), _stream(stream)))


def csgmv_build_lm_head_batch_info(bi: BatchInfo, pruned_lens: torch.Tensor, req_adapter: torch.Tensor,
                                   num_tokens: int, lora_ranks: torch.Tensor, scalings: torch.Tensor,
                                   max_chunk_size: int = 128, chunk_size_override: int = 0,
                                   use_cuda_graph: bool = False, stream=None) -> None:
    bs = int(pruned_lens.numel())
    _check(lib().csgmv_build_lm_head_batch_info(ctypes.byref(bi.c), _ptr(pruned_lens), _ptr(req_adapter), bs,
                                                int(num_tokens), _ptr(lora_ranks), _ptr(scalings),
                                                int(lora_ranks.numel()), int(max_chunk_size),
                                                int(chunk_size_override), int(bool(use_cuda_graph)),
                                                _stream(stream)))


def csgmv_shrink(x: torch.Tensor, A: torch.Tensor, num_slices: int, h: torch.Tensor, bi: BatchInfo,
                 stream=None) -> torch.Tensor:
    s, K = x.shape
    dt = CSGMV_DTYPE_F32 if h.dtype == torch.float32 else CSGMV_DTYPE_BF16
    _check(lib().csgmv_shrink(_ptr(x), int(s), int(K), _ptr(A), int(num_slices), _ptr(h), dt,
                              int(h.stride(0)), ctypes.byref(bi.c), _stream(stream)))
    return h


def csgmv_expand(h: torch.Tensor, B: torch.Tensor, slice_offsets, num_slices: int, max_slice_size: int,
                 out: torch.Tensor, accumulate: bool, bi: BatchInfo, stream=None) -> torch.Tensor:
    dt = CSGMV_DTYPE_F32 if h.dtype == torch.float32 else CSGMV_DTYPE_BF16
    N = int(out.shape[1])
    _check(lib().csgmv_expand(_ptr(h), dt, int(h.stride(0)), _ptr(B), N, _offsets(slice_offsets),
                              int(num_slices), int(max_slice_size), _ptr(out), int(bool(accumulate)),
                              ctypes.byref(bi.c), _stream(stream)))
    return out


def csgmv_qkv(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, slice_offsets, num_slices: int,
              max_slice_size: int, base_output: torch.Tensor, bi: BatchInfo, stream=None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    K = int(x.shape[1])
    N = int(base_output.shape[1])
    ws = _ptr(workspace) if workspace is not None else None
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().csgmv_qkv(_ptr(x), K, _ptr(A), _ptr(B), N, _offsets(slice_offsets), int(num_slices),
                           int(max_slice_size), _ptr(base_output), ws, wsb, ctypes.byref(bi.c), _stream(stream)))
    return base_output


def csgmv_qkv_path(bi: BatchInfo, K: int, N: int, slice_offsets, num_slices: int, workspace_bytes: int) -> str:
    """Which kernels csgmv_qkv runs for the batch last built into bi: "fused"
    (one kernel) or a two-kernel path ("decode", "small_split", "stream").
    Host only."""
    rc = lib().csgmv_qkv_path(ctypes.byref(bi.c), int(K), int(N), _offsets(slice_offsets), int(num_slices),
                              int(workspace_bytes))
    if rc < 0:
        _check(rc)
    return PATHS[rc]


def csgmv_qkv_workspace_bytes(bi: BatchInfo, num_slices: int) -> int:
    return int(lib().csgmv_qkv_workspace_bytes(ctypes.byref(bi.c), int(num_slices)))


def csgmv_qkv_static_scratch(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, slice_offsets, num_slices: int,
                             max_slice_size: int, base_output: torch.Tensor, bi: BatchInfo,
                             stream=None) -> torch.Tensor:
    """csgmv_qkv with the library's own fixed device scratch for h, for
    callers that cannot allocate a workspace (see csgmv.h)."""
    K = int(x.shape[1])
    N = int(base_output.shape[1])
    _check(lib().csgmv_qkv_static_scratch(_ptr(x), K, _ptr(A), _ptr(B), N, _offsets(slice_offsets),
                                          int(num_slices), int(max_slice_size), _ptr(base_output),
                                          ctypes.byref(bi.c), _stream(stream)))
    return base_output


def embedding_lora_a(input_ids: torch.Tensor, A_emb: torch.Tensor, vocab_size: int, out: torch.Tensor,
                     bi: BatchInfo, stream=None) -> torch.Tensor:
    rank = int(out.shape[1])
    _check(lib().embedding_lora_a(_ptr(input_ids), _ptr(A_emb), int(vocab_size), rank, _ptr(out),
                                  ctypes.byref(bi.c), _stream(stream)))
    return out


def embedding_lora_a_extra(input_ids: torch.Tensor, A_emb: torch.Tensor, vocab_size: int,
                           extra_embeddings: torch.Tensor | None, out: torch.Tensor, bi: BatchInfo,
                           stream=None) -> torch.Tensor:
    """out (s, R) = LoRA-A rows of each token's id, from A_emb (L, R, V) for
    ids below vocab_size and from extra_embeddings (L, E, R) above."""
    E = 0 if extra_embeddings is None else int(extra_embeddings.shape[1])
    _check(lib().embedding_lora_a_extra(_ptr(input_ids), _ptr(A_emb), int(vocab_size), int(out.shape[1]),
                                        _ptr(extra_embeddings), E, _ptr(out), ctypes.byref(bi.c), _stream(stream)))
    return out


def embedding_lora_a_transposed(input_ids: torch.Tensor, A_emb_t: torch.Tensor, vocab_size: int,
                                extra_embeddings: torch.Tensor | None, out: torch.Tensor, bi: BatchInfo,
                                stream=None) -> torch.Tensor:
    """embedding_lora_a_extra with the table stored as A_emb_t (L, V, R)."""
    E = 0 if extra_embeddings is None else int(extra_embeddings.shape[1])
    _check(lib().embedding_lora_a_transposed(_ptr(input_ids), _ptr(A_emb_t), int(vocab_size), int(out.shape[1]),
                                             _ptr(extra_embeddings), E, _ptr(out), ctypes.byref(bi.c),
                                             _stream(stream)))
    return out


def csgmv_transpose_embedding(A_emb: torch.Tensor, A_emb_t: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """A_emb_t (L, V, R) from A_emb (L, R, V), on the device (load time)."""
    L, R, V = (int(v) for v in A_emb.shape)
    if A_emb_t is None:
        A_emb_t = torch.empty((L, V, R), dtype=A_emb.dtype, device=A_emb.device)
    _check(lib().csgmv_transpose_embedding(_ptr(A_emb), L, R, V, _ptr(A_emb_t), _stream(stream)))
    return A_emb_t


def extra_token_embedding(input_ids: torch.Tensor, output: torch.Tensor, extra_embeddings: torch.Tensor,
                          vocab_size: int, bi: BatchInfo, stream=None) -> torch.Tensor:
    """Rows of extra tokens (ids >= vocab_size) of output (s, D) become
    extra_embeddings[slot][id - vocab_size]; other rows are untouched."""
    _check(lib().extra_token_embedding(_ptr(input_ids), _ptr(output), int(output.shape[1]), _ptr(extra_embeddings),
                                       int(extra_embeddings.shape[1]), int(vocab_size), ctypes.byref(bi.c),
                                       _stream(stream)))
    return output


def _slice_ptrs(B_slices) -> ctypes.Array:
    return (ctypes.c_void_p * len(B_slices))(*[t.data_ptr() for t in B_slices])


def csgmv_expand_sliced(h: torch.Tensor, B_slices, slice_offsets, num_slices: int, max_slice_size: int,
                        out: torch.Tensor, accumulate: bool, bi: BatchInfo, stream=None) -> torch.Tensor:
    """csgmv_expand with B given per slice: B_slices[j] is (max_loras, off[j+1]-off[j], R)."""
    dt = CSGMV_DTYPE_F32 if h.dtype == torch.float32 else CSGMV_DTYPE_BF16
    _check(lib().csgmv_expand_sliced(_ptr(h), dt, int(h.stride(0)), _slice_ptrs(B_slices), int(out.shape[1]),
                                     _offsets(slice_offsets), int(num_slices), int(max_slice_size), _ptr(out),
                                     int(bool(accumulate)), ctypes.byref(bi.c), _stream(stream)))
    return out


def csgmv_qkv_sliced(x: torch.Tensor, A: torch.Tensor, B_slices, slice_offsets, num_slices: int,
                     max_slice_size: int, base_output: torch.Tensor, bi: BatchInfo, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """csgmv_qkv with B given per slice (the tuple form of run_qkv_lora /
    run_gate_up_lora): B_slices[j] is (max_loras, off[j+1]-off[j], R)."""
    K = int(x.shape[1])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().csgmv_qkv_sliced(_ptr(x), K, _ptr(A), _slice_ptrs(B_slices), int(base_output.shape[1]),
                                  _offsets(slice_offsets), int(num_slices), int(max_slice_size), _ptr(base_output),
                                  _ptr(workspace), ws_bytes, ctypes.byref(bi.c), _stream(stream)))
    return base_output


# ---------------------------------------------------------------------------
# The serving step around the adapters: paged K/V cache, attention of draft
# trees, draft verification (include/csgmv.h has each call's contract).

_KV_DTYPES = {torch.bfloat16: CSGMV_DTYPE_BF16, torch.float16: CSGMV_DTYPE_F16}


def _need(ok: bool, msg: str):
    """Checks that only the binding can make (a tensor's type and shape, which
    the C ABI does not see) fail as the library's own argument checks do.
    (Where a call's latency counts, a message is put together only when it is
    raised.)"""
    if not ok:
        raise CsgmvError(-1, msg)


def _need_i32(device: int, name: str, t: torch.Tensor | None, *shape):
    """t is a dense int32 tensor on that GPU, of that shape (None: any extent)."""
    if t is not None and (t.dtype is not torch.int32 or t.get_device() != device or not t.is_contiguous() or
                          not _has_shape(t.shape, shape)):
        raise CsgmvError(-1, f"{name} must be a contiguous int32 tensor of shape {shape} on cuda:{device}, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_f32(device: int, name: str, t: torch.Tensor, *shape):
    if t.dtype is not torch.float32 or t.get_device() != device or not _has_shape(t.shape, shape):
        raise CsgmvError(-1, f"{name} must be a float32 tensor of shape {shape} on cuda:{device}, "
                             f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _has_shape(have, want) -> bool:
    return have == want or (len(have) == len(want) and all(w is None or w == n for n, w in zip(have, want)))


def _at(t: torch.Tensor | None):
    """t's address, as the calls take it."""
    return None if t is None else t.data_ptr()


# torch.cuda.current_stream() builds an object (3 us); the handle alone is a lookup
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device: int):
    """The CUDA stream handle to launch on: stream, or the device's current one.
    The library launches on the current device, so that has to be the operands'
    (a handle does not say: the default stream's is 0 on every device)."""
    if torch.cuda.current_device() != device:
        raise CsgmvError(-1, f"the operands are on cuda:{device}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is not None:
        at = getattr(stream, "device_index", device)  # (a bare handle's holder need not say)
        if at != device:
            raise CsgmvError(-1, f"the operands are on cuda:{device}, the stream is on cuda:{at}")
        return stream.cuda_stream
    if _current_raw_stream is not None:
        return _current_raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


def _empty(stream, *size, **kw) -> torch.Tensor:
    """torch.empty for a call on `stream` (None: the current one).  The memory
    belongs to that stream: another one's could still be in use by what was
    put on that one before, and be given out again there while the call runs."""
    if stream is None:
        return torch.empty(*size, **kw)
    with torch.cuda.stream(stream):
        return torch.empty(*size, **kw)


def _alike(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Same shape and the same strides where they matter."""
    return a.shape == b.shape and (a.stride() == b.stride() or a.numel() == 0 or all(
        n <= 1 or x == y for n, x, y in zip(a.shape, a.stride(), b.stride())))


class KvCache:
    """A paged K/V cache over caller-owned tensors, and the C struct that
    points at them.

      k_pages, v_pages   bf16 or f16, (layers, pages, kv_heads, page_size, head_dim)
                         ("HND") or (layers, pages, page_size, kv_heads, head_dim)
                         ("NHD"); any strides that are multiples of 8, the last 1
      page_table         int32 (max_seqs, max_pages_per_seq), -1 where empty
      seq_lens           int32 (max_seqs,)
      page_refs          int32 (pages,)

    KvCache.allocate() makes an empty cache with its own tensors."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                 page_refs: torch.Tensor, layout: str = "HND"):
        _need(layout in ("HND", "NHD"), f"layout {layout!r} must be HND or NHD")
        _need(k_pages.dtype in _KV_DTYPES and v_pages.dtype == k_pages.dtype, "k_pages / v_pages must be bf16 or f16, both alike")
        _need(k_pages.dim() == 5 and _alike(k_pages, v_pages),
              "k_pages / v_pages must have five dimensions and the same shape and strides")
        _need(k_pages.is_cuda and v_pages.get_device() == k_pages.get_device(),
              "k_pages / v_pages must be CUDA tensors on one device")
        _need(k_pages.stride(4) == 1, "the last dimension of k_pages / v_pages must be dense")
        h, t = (2, 3) if layout == "HND" else (3, 2)
        layers, pages, heads, ps, d = (int(k_pages.shape[i]) for i in (0, 1, h, t, 4))
        at = k_pages.get_device()
        _need(page_table.dim() == 2, "page_table must have two dimensions")
        seqs, max_pages = (int(n) for n in page_table.shape)
        _need_i32(at, "page_table", page_table, seqs, max_pages)
        _need_i32(at, "seq_lens", seq_lens, seqs)
        _need_i32(at, "page_refs", page_refs, pages)
        self.k_pages, self.v_pages = k_pages, v_pages
        self.page_table, self.seq_lens, self.page_refs = page_table, seq_lens, page_refs
        self.layout = layout
        dev = k_pages.device
        self.scratch = torch.empty(csgmv_kv_scratch_ints(pages, seqs), dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        c = _KvCacheC()
        for n in ("k_pages", "v_pages", "page_table", "seq_lens", "page_refs", "scratch", "status"):
            setattr(c, n, getattr(self, n).data_ptr())
        c.token_stride, c.head_stride = int(k_pages.stride(t)), int(k_pages.stride(h))
        c.page_stride, c.layer_stride = int(k_pages.stride(1)), int(k_pages.stride(0))
        c.dtype, c.num_layers, c.num_pages, c.page_size = _KV_DTYPES[k_pages.dtype], layers, pages, ps
        c.num_kv_heads, c.head_dim, c.max_seqs, c.max_pages_per_seq = heads, d, seqs, max_pages
        self.c = c
        self._ref = ctypes.byref(c)
        self.dtype, self.device = k_pages.dtype, at
        self.num_layers, self.num_pages, self.page_size = layers, pages, ps
        self.num_kv_heads, self.head_dim, self.max_seqs, self.max_pages_per_seq = heads, d, seqs, max_pages
        self.row_shape = (heads, d)

    @classmethod
    def allocate(cls, num_layers: int, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
                 max_seqs: int, max_pages_per_seq: int, dtype=torch.bfloat16, layout: str = "HND", device="cuda"):
        """An empty cache with tensors of its own."""
        shape = ((num_layers, num_pages, num_kv_heads, page_size, head_dim) if layout == "HND" else
                 (num_layers, num_pages, page_size, num_kv_heads, head_dim))
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device),
                   torch.full((max_seqs, max_pages_per_seq), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(num_pages, **i32), layout=layout)

    def with_lens(self, seq_lens: torch.Tensor) -> "KvCache":
        """The same cache (pages, table, counts, scratch, status) seen with other
        lengths, e.g. those before csgmv_kv_extend: for calls that read it."""
        _need_i32(self.device, "seq_lens", seq_lens, self.max_seqs)
        other = object.__new__(KvCache)
        other.__dict__.update(self.__dict__)
        other.seq_lens = seq_lens
        other.c = _KvCacheC()
        ctypes.pointer(other.c)[0] = self.c
        other.c.seq_lens = seq_lens.data_ptr()
        other._ref = ctypes.byref(other.c)
        return other

    def device_status(self) -> int:
        return int(self.status.item())


def csgmv_kv_scratch_ints(num_pages: int, max_seqs: int) -> int:
    return int(lib().csgmv_kv_scratch_ints(int(num_pages), int(max_seqs)))


def _new_rows(cache: KvCache, k_new: torch.Tensor, v_new: torch.Tensor, lead: tuple):
    """k_new / v_new are (*lead, kv_heads, head_dim) in the cache's type; their strides."""
    st, want = k_new.stride(), lead + cache.row_shape
    if k_new.shape != want or st[-1] != 1:
        raise CsgmvError(-1, f"k_new / v_new must be {want} (the cache's layers, kv_heads and head_dim), the last "
                             f"dimension dense, not {tuple(k_new.shape)}")
    if v_new.shape != want or v_new.stride() != st and not _alike(k_new, v_new):
        raise CsgmvError(-1, "k_new / v_new must have the same shape and strides")
    if not (k_new.dtype is v_new.dtype is cache.dtype and k_new.get_device() == v_new.get_device() == cache.device):
        raise CsgmvError(-1, "k_new / v_new must be CUDA tensors of the cache's type, on its device")
    return st


def csgmv_kv_commit(cache: KvCache, k_new: torch.Tensor, v_new: torch.Tensor, accept_index: torch.Tensor | None,
                    accept_len: torch.Tensor, tree_indptr: torch.Tensor, seq_slots: torch.Tensor | None = None,
                    stream=None) -> None:
    """Appends accept_len[b] of request b's rows of k_new / v_new (layers,
    tokens, kv_heads, head_dim) to its sequence: rows tree_indptr[b] +
    accept_index[b, j], or its first rows without an accept_index."""
    st = _new_rows(cache, k_new, v_new, (cache.num_layers, k_new.shape[1]))
    bs = accept_len.numel()
    width = 0 if accept_index is None else accept_index.shape[-1]
    _need_i32(cache.device, "accept_len", accept_len, bs)
    if accept_index is not None:
        _need_i32(cache.device, "accept_index", accept_index, bs, width)
    _need_i32(cache.device, "tree_indptr", tree_indptr, bs + 1)
    if seq_slots is not None:
        _need_i32(cache.device, "seq_slots", seq_slots, bs)
    rc = lib().csgmv_kv_commit(cache._ref, k_new.data_ptr(), v_new.data_ptr(), st[0], st[1], st[2], k_new.shape[1],
                               _at(accept_index), width, accept_len.data_ptr(), tree_indptr.data_ptr(),
                               _at(seq_slots), bs, _raw_stream(stream, cache.device))
    if rc:
        _check(rc)


def csgmv_kv_fork(cache: KvCache, parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
    """Sequence children[i] becomes a copy of sequence parents[i]."""
    n = parents.numel()
    _need_i32(cache.device, "parents", parents, n)
    _need_i32(cache.device, "children", children, n)
    _check(lib().csgmv_kv_fork(cache._ref, parents.data_ptr(), children.data_ptr(), n,
                               _raw_stream(stream, cache.device)))


def csgmv_kv_free(cache: KvCache, seqs: torch.Tensor, keep_lens: torch.Tensor | None = None, stream=None) -> None:
    """Cuts sequence seqs[i] back to keep_lens[i] tokens (None: to nothing)."""
    n = seqs.numel()
    _need_i32(cache.device, "seqs", seqs, n)
    _need_i32(cache.device, "keep_lens", keep_lens, n)
    _check(lib().csgmv_kv_free(cache._ref, seqs.data_ptr(), _at(keep_lens), n, _raw_stream(stream, cache.device)))


def csgmv_kv_compact(cache: KvCache, stream=None) -> None:
    """Moves live pages into the holes below them; live pages end up first."""
    _check(lib().csgmv_kv_compact(cache._ref, _raw_stream(stream, cache.device)))


def csgmv_kv_copy_pages(cache: KvCache, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Copies the contents of pages src[i] to pages dst[i] in every layer."""
    n = src.numel()
    _need_i32(cache.device, "src", src, n)
    _need_i32(cache.device, "dst", dst, n)
    _check(lib().csgmv_kv_copy_pages(cache._ref, src.data_ptr(), dst.data_ptr(), n, _raw_stream(stream, cache.device)))


def csgmv_tree_attention_workspace_bytes(cache: KvCache, num_q_heads: int) -> int:
    return int(lib().csgmv_tree_attention_workspace_bytes(cache._ref, int(num_q_heads)))


def csgmv_tree_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: KvCache, layer: int,
                         tree_indptr: torch.Tensor, out: torch.Tensor, mask: torch.Tensor | None = None,
                         seq_slots: torch.Tensor | None = None, scale: float | None = None,
                         lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Attention of request b's rows of q (tokens, heads, head_dim) over its
    cached sequence and over its own rows of k_new / v_new that `mask` (int32
    bits, (tokens, words); None: causal) lets each row see.  scale defaults to
    head_dim ** -0.5; lse (tokens, heads) f32 is optional.  A workspace that is
    not given is allocated on the call's stream."""
    shape, qs, os_ = q.shape, q.stride(), out.stride()
    if len(shape) != 3 or out.shape != shape:
        raise CsgmvError(-1, "q and out must be (tokens, heads, head_dim)")
    if not (q.dtype is out.dtype is cache.dtype and q.get_device() == out.get_device() == cache.device):
        raise CsgmvError(-1, "q and out must be CUDA tensors of the cache's type, on its device")
    n, hq, d = shape
    if d != cache.head_dim or n and (qs[2] != 1 or os_[2] != 1):
        raise CsgmvError(-1, "q and out must have the cache's head_dim, dense")
    ks = _new_rows(cache, k_new, v_new, (n,))
    bs, words = tree_indptr.shape[0] - 1 if tree_indptr.dim() else 0, 0
    _need_i32(cache.device, "tree_indptr", tree_indptr, bs + 1)
    if mask is not None:
        words = mask.shape[-1]
        _need_i32(cache.device, "mask", mask, n, words)
    if seq_slots is not None:
        _need_i32(cache.device, "seq_slots", seq_slots, bs)
    if lse is not None:
        _need_f32(cache.device, "lse", lse, n, hq)
        if not lse.is_contiguous():
            raise CsgmvError(-1, "lse must be contiguous")
    if workspace is None:
        workspace = _empty(stream, csgmv_tree_attention_workspace_bytes(cache, hq), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != cache.device or not workspace.is_contiguous():
        raise CsgmvError(-1, "the workspace must be a contiguous tensor on the cache's device")
    rc = lib().csgmv_tree_attention(
        q.data_ptr(), qs[0], qs[1], hq, k_new.data_ptr(), v_new.data_ptr(), ks[0], ks[1], cache._ref, layer,
        tree_indptr.data_ptr(), _at(seq_slots), bs, n, _at(mask), words, d ** -0.5 if scale is None else scale,
        out.data_ptr(), os_[0], os_[1], _at(lse), workspace.data_ptr(), workspace.nbytes,
        _raw_stream(stream, cache.device))
    if rc:
        _check(rc)
    return out


class DraftTree:
    """Device buffers of csgmv_build_draft_tree for up to max_nodes drafted
    tokens, with at most max_draft of them in one request."""

    def __init__(self, max_nodes: int, max_draft: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.words = max(1, (int(max_draft) + 31) // 32)
        self.max_draft = int(max_draft)
        self.mask = torch.zeros((max_nodes, self.words), **i32)
        self.depth = torch.zeros(max_nodes, **i32)
        self.first_child = torch.full((max_nodes,), -1, **i32)
        self.next_sibling = torch.full((max_nodes,), -1, **i32)
        self.status = torch.zeros(1, **i32)
        self.max_nodes, self.device = int(max_nodes), self.status.get_device()
        self._at = tuple(t.data_ptr() for t in (self.mask, self.depth, self.first_child, self.next_sibling, self.status))

    def device_status(self) -> int:
        return int(self.status.item())


def csgmv_build_draft_tree(tree: DraftTree, parents: torch.Tensor, tree_indptr: torch.Tensor, stream=None) -> None:
    """Fills tree.mask, depth, first_child and next_sibling from the nodes'
    parents (numbers inside their request, -1 at its node 0)."""
    n, bs = parents.numel(), tree_indptr.numel() - 1
    _need_i32(tree.device, "parents", parents, n)
    _need_i32(tree.device, "tree_indptr", tree_indptr, bs + 1)
    if n > tree.max_nodes:
        raise CsgmvError(-1, f"{n} nodes exceed the tree's {tree.max_nodes}")
    rc = lib().csgmv_build_draft_tree(parents.data_ptr(), tree_indptr.data_ptr(), bs, n, tree.words, *tree._at,
                                      _raw_stream(stream, tree.device))
    if rc:
        _check(rc)


def csgmv_verify_drafts(target_probs: torch.Tensor, draft_tokens: torch.Tensor, tree_indptr: torch.Tensor,
                        tree: DraftTree, accept_uniforms: torch.Tensor, sample_uniforms: torch.Tensor,
                        draft_probs: torch.Tensor | None = None, accept_index: torch.Tensor | None = None,
                        accept_len: torch.Tensor | None = None, next_token: torch.Tensor | None = None, stream=None):
    """Walks each tree: (accept_index (bs, width), accept_len (bs,), next_token
    (bs,)), allocated (on the call's stream) unless given; width defaults to
    tree.max_draft.
    draft_probs None: the drafts were chosen, not sampled."""
    n, bs = draft_tokens.numel(), tree_indptr.numel() - 1
    _need_f32(tree.device, "target_probs", target_probs, n, None)
    ts, vocab = target_probs.stride(), target_probs.shape[1]
    if n and ts[1] != 1:
        raise CsgmvError(-1, "target_probs must have dense rows")
    # the row stride of a single row says nothing
    ts, ds = ts[0] if n > 1 else vocab, 0
    if draft_probs is not None:
        _need_f32(tree.device, "draft_probs", draft_probs, n, vocab)
        ds = draft_probs.stride()
        if n and ds[1] != 1:
            raise CsgmvError(-1, "draft_probs must have dense rows")
        ds = ds[0] if n > 1 else vocab
    _need_i32(tree.device, "draft_tokens", draft_tokens, n)
    _need_i32(tree.device, "tree_indptr", tree_indptr, bs + 1)
    _need_f32(tree.device, "accept_uniforms", accept_uniforms, n)
    _need_f32(tree.device, "sample_uniforms", sample_uniforms, bs)
    if not (accept_uniforms.is_contiguous() and sample_uniforms.is_contiguous()):
        raise CsgmvError(-1, "the uniform numbers must be contiguous")
    if n > tree.max_nodes:
        raise CsgmvError(-1, f"{n} nodes exceed the tree's {tree.max_nodes}")
    width = tree.max_draft if accept_index is None else accept_index.shape[-1]
    if accept_index is None and accept_len is None and next_token is None:  # one buffer for all
        accept_index, accept_len, next_token = _empty(
            stream, bs * (width + 2), dtype=torch.int32, device=target_probs.device).split_with_sizes([bs * width, bs, bs])
        accept_index = accept_index.view(bs, width)
    else:
        new = dict(dtype=torch.int32, device=target_probs.device)
        accept_index = _empty(stream, (bs, width), **new) if accept_index is None else accept_index
        accept_len = _empty(stream, bs, **new) if accept_len is None else accept_len
        next_token = _empty(stream, bs, **new) if next_token is None else next_token
        _need_i32(tree.device, "accept_index", accept_index, bs, width)
        _need_i32(tree.device, "accept_len", accept_len, bs)
        _need_i32(tree.device, "next_token", next_token, bs)
    rc = lib().csgmv_verify_drafts(
        target_probs.data_ptr(), ts, _at(draft_probs), ds, draft_tokens.data_ptr(), tree_indptr.data_ptr(), tree._at[2],
        tree._at[3], accept_uniforms.data_ptr(), sample_uniforms.data_ptr(), bs, n, vocab, accept_index.data_ptr(), width,
        accept_len.data_ptr(), next_token.data_ptr(), tree._at[4], _raw_stream(stream, tree.device))
    if rc:
        _check(rc)
    return accept_index, accept_len, next_token


# ---------------------------------------------------------------------------
# What a decoder does between the projections, the attention and the
# verification: residual and norms, rotary positions, appending to the cache
# layer by layer, logits to probabilities.

_DTYPES = {torch.bfloat16: CSGMV_DTYPE_BF16, torch.float16: CSGMV_DTYPE_F16, torch.float32: CSGMV_DTYPE_F32}
NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}


class Norm:
    """A norm over rows of `hidden` elements, and the C struct of it: kind "rms"
    or "layer", weight and bias dense vectors of the rows' type or None."""

    def __init__(self, kind: str = "rms", weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                 eps: float = 1e-6):
        _need(kind in NORM_KINDS, f"kind {kind!r} must be one of {', '.join(NORM_KINDS)}")
        of = [t for t in (weight, bias) if t is not None]
        _need(all(t.is_cuda and t.dim() == 1 and t.is_contiguous() for t in of),
              "a norm's weight and bias must be dense CUDA vectors")
        _need(len(of) < 2 or (of[0].shape == of[1].shape and of[0].dtype is of[1].dtype and of[0].device == of[1].device),
              "a norm's weight and bias must be alike")
        self.kind, self.weight, self.bias, self.eps = kind, weight, bias, eps
        self.hidden = of[0].shape[0] if of else None
        self.dtype = of[0].dtype if of else None
        self.device = of[0].get_device() if of else None
        self.c = _NormC(_at(weight), _at(bias), eps, NORM_KINDS[kind])
        self._ref = ctypes.byref(self.c)


def _norm_for(norm: Norm | None, x: torch.Tensor, hidden: int):
    if norm is None:
        return None
    if norm.hidden is not None and not (norm.hidden == hidden and norm.dtype is x.dtype and norm.device == x.get_device()):
        raise CsgmvError(-1, f"a norm's weight is {norm.dtype} ({norm.hidden},) on cuda:{norm.device}, the rows are {x.dtype} "
                             f"of {hidden} on {x.device}")
    return norm._ref


def _row_stride(name: str, t: torch.Tensor, n: int, hidden: int, device: int) -> int:
    """t is (n, hidden) on that GPU, its rows dense; their stride."""
    st = t.stride()
    if t.shape != (n, hidden) or t.get_device() != device or hidden > 1 and st[1] != 1:
        raise CsgmvError(-1, f"{name} must be ({n}, {hidden}) on cuda:{device}, its rows dense, not {tuple(t.shape)} on {t.device}")
    return st[0] if n > 1 else hidden


def csgmv_add_norm(x: torch.Tensor, norm: Norm | None, out: torch.Tensor | None = None,
                   residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                   post_norm: Norm | None = None, gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                   stream=None) -> torch.Tensor | None:
    """r' = residual_scale * residual + gate * post_norm(x); out = norm(r').

    x, out and gate (tokens, hidden) in one type (gate may be a single row);
    residual in that type or f32.  residual_out None: the residual is updated in
    place (without one, r' is not kept).  out None: allocated on the call's
    stream, unless norm is None too: then only r' is made."""
    if x.dim() != 2 or x.dtype not in _DTYPES or not x.is_cuda:
        raise CsgmvError(-1, "x must be a CUDA tensor (tokens, hidden) of bf16, f16 or f32")
    n, hidden = x.shape
    device, rtype = x.get_device(), x.dtype
    xs, rs, ros, gs, os_ = _row_stride("x", x, n, hidden, device), 0, 0, 0, 0
    if residual is not None:
        rtype = residual.dtype
        rs = _row_stride("residual", residual, n, hidden, device)
        if residual_out is None:
            residual_out = residual
    if residual_out is not None:
        ros = _row_stride("residual_out", residual_out, n, hidden, device)
        if residual is None:
            rtype = residual_out.dtype
        elif residual_out.dtype is not rtype:
            raise CsgmvError(-1, "residual_out must have the residual's type")
    if rtype is not x.dtype and rtype is not torch.float32:
        raise CsgmvError(-1, f"the residual must be {x.dtype} or float32, not {rtype}")
    if gate is not None:
        if gate.dtype is not x.dtype:
            raise CsgmvError(-1, f"gate must be {x.dtype}, not {gate.dtype}")
        one = gate.shape[0] == 1
        gs = _row_stride("gate", gate, 1 if one else n, hidden, device)
        if one:
            gs = 0
    if out is None:
        if norm is not None:
            out = _empty(stream, (n, hidden), dtype=x.dtype, device=x.device)
            os_ = hidden
    else:
        if out.dtype is not x.dtype:
            raise CsgmvError(-1, f"out must be {x.dtype}, not {out.dtype}")
        os_ = _row_stride("out", out, n, hidden, device)
    rc = lib().csgmv_add_norm(x.data_ptr(), xs, _DTYPES[x.dtype], _at(residual), rs, _DTYPES[rtype], _at(gate), gs,
                              _norm_for(post_norm, x, hidden), _norm_for(norm, x, hidden), residual_scale, n, hidden,
                              _at(residual_out), ros, _at(out), os_, _raw_stream(stream, device))
    if rc:
        _check(rc)
    return out


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: tuple | None = None):
    """(radians a position of each pair, float64 on the CPU; the factor of the
    turned part) of rotary positions: base ** (-2 i / rotary_dim), stretched for
    contexts longer than the trained one by scaling:

      ("linear", factor)      every angle divided by factor
      ("ntk", factor)         base * factor ** (rotary_dim / (rotary_dim - 2)) in
                              place of base
      ("wavelength", factor, low, high, original)
                              a pair that makes fewer than low turns in the original
                              context is divided by factor, one that makes more than
                              high is kept, others are blended in between
      ("yarn", factor, original[, fast = 32, slow = 1])
                              pairs from the one that makes `fast` turns in the
                              original context to the one that makes `slow` are
                              blended along their index (the ramp may end behind
                              the last pair, at rotary_dim - 1 at most); the turned
                              part is multiplied by 0.1 ln(factor) + 1"""
    _need(rotary_dim >= 0 and rotary_dim % 2 == 0, f"rotary_dim {rotary_dim} must be even and not negative")
    _need(0 < base < math.inf, "base must be positive and finite")
    n = rotary_dim // 2
    i = torch.arange(n, dtype=torch.float64)
    if n == 0:
        return i, 1.0
    f = base ** (-2.0 * i / rotary_dim)
    if scaling is None:
        return f, 1.0
    kind, more = scaling[0], scaling[1:]
    lengths = {"linear": (1,), "ntk": (1,), "wavelength": (4,), "yarn": (2, 4)}
    _need(kind in lengths and len(more) in lengths[kind] and all(0 < v < math.inf for v in more),
          f"scaling {scaling!r} is none of those that are known, or not positive and finite")
    factor = float(more[0])
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ntk":
        _need(rotary_dim > 2, "ntk scaling needs a rotary_dim above 2")
        return (base * factor ** (rotary_dim / (rotary_dim - 2.0))) ** (-2.0 * i / rotary_dim), 1.0
    if kind == "wavelength":
        _, low, high, original = more
        _need(high > low, "wavelength scaling needs low < high")
        keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 1.0
    original, (fast, slow) = more[1], more[2:] or (32.0, 1.0)
    _need(base > 1.0 and fast >= slow, "yarn scaling needs a base above 1 and fast >= slow")

    def pair(turns):
        return rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rotary_dim - 1)
    blend = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
    return f * (1 - blend) + f / factor * blend, 0.1 * math.log(factor) + 1.0


def csgmv_rope_turns(freq) -> torch.Tensor:
    """Frequencies (radians a position) in 2^-64 turns, as an int64 tensor that
    holds the unsigned numbers' bits."""
    freq = torch.as_tensor(freq, dtype=torch.float64).cpu().contiguous()
    turns = torch.empty(freq.shape, dtype=torch.int64)
    _check(lib().csgmv_rope_turns(freq.data_ptr(), freq.numel(), turns.data_ptr()))
    return turns


class Rope:
    """Rotary positions of heads of head_dim: the first rotary_dim elements
    (None: all), pairs (2 i, 2 i + 1) if interleaved, else (i, i + rotary_dim / 2).
    freq (radians a position of each pair) and scale take the place of what
    rope_frequencies(rotary_dim, base, scaling) gives."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: tuple | None = None, freq=None, scale: float | None = None, device="cuda"):
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        _need(rotary_dim <= head_dim, f"rotary_dim {rotary_dim} exceeds head_dim {head_dim}")
        own, factor = rope_frequencies(rotary_dim, base, scaling)
        self.freq = own if freq is None else torch.as_tensor(freq, dtype=torch.float64).cpu()
        _need(self.freq.shape == own.shape, f"freq must have {rotary_dim // 2} entries")
        self.scale = factor if scale is None else scale
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, rotary_dim, bool(interleaved)
        self.turns = csgmv_rope_turns(self.freq).to(device)
        _need(self.turns.is_cuda, "a rope's device must be a CUDA device")
        self.device = self.turns.get_device()
        self.c = _RopeC(self.turns.data_ptr(), self.scale, rotary_dim, int(interleaved))
        self._ref = ctypes.byref(self.c)


def _head_strides(name: str, t: torch.Tensor, n: int, heads, d: int, dtype, device: int):
    """t is (n, heads, d) in that type on that GPU, its heads dense; its strides."""
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != n or heads is not None and shape[1] != heads or shape[2] != d or \
            t.dtype is not dtype or t.get_device() != device or n and d > 1 and st[2] != 1:
        raise CsgmvError(-1, f"{name} must be ({n}, {'heads' if heads is None else heads}, {d}) of {dtype} on cuda:{device}, "
                             f"its heads dense, not {tuple(shape)} of {t.dtype} on {t.device}")
    return st


def csgmv_rotary(rope: Rope, positions: torch.Tensor, q: torch.Tensor, k: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, inverse: bool = False, stream=None):
    """q and k (tokens, heads, head_dim; bf16, f16 or f32) turned by positions
    (int32, (tokens,)) into q_out and k_out (None: in place); returns those.
    inverse: by the negative angles (the gradient of the inputs from that of the
    outputs)."""
    n, d, dtype, device = q.shape[0], rope.head_dim, q.dtype, rope.device
    if dtype not in _DTYPES:
        raise CsgmvError(-1, f"q must be bf16, f16 or f32, not {dtype}")
    _need_i32(device, "positions", positions, n)
    qs = _head_strides("q", q, n, None, d, dtype, device)
    hq, hk = q.shape[1], 0
    if q_out is None or q_out is q:
        q_out, qos = q, qs
    else:
        qos = _head_strides("q_out", q_out, n, hq, d, dtype, device)
    if k is None:
        if k_out is not None:
            raise CsgmvError(-1, "k_out without k")
        ks = kos = (0, 0)
    else:
        ks = _head_strides("k", k, n, None, d, dtype, device)
        hk = k.shape[1]
        if k_out is None or k_out is k:
            k_out, kos = k, ks
        else:
            kos = _head_strides("k_out", k_out, n, hk, d, dtype, device)
    rc = lib().csgmv_rotary(rope._ref, _DTYPES[dtype], d, positions.data_ptr(), n, q.data_ptr(), qs[0], qs[1], hq, _at(k), ks[0],
                            ks[1], hk, q_out.data_ptr(), qos[0], qos[1], _at(k_out), kos[0], kos[1], inverse,
                            _raw_stream(stream, device))
    if rc:
        _check(rc)
    return q_out, k_out


def csgmv_kv_extend(cache: KvCache, tree_indptr: torch.Tensor, num_tokens: int, add_lens: torch.Tensor | None = None,
                    seq_slots: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                    positions: torch.Tensor | None = None, lens_before: torch.Tensor | None = None, stream=None):
    """Room for add_lens[b] (None: all) of request b's rows of a batch of
    num_tokens rows in its sequence: (slots int64, positions int32), one of each a
    row, allocated on the call's stream unless given.  lens_before (int32,
    (max_seqs,)) gets the lengths as they were (KvCache.with_lens)."""
    device = cache.device
    bs = tree_indptr.shape[0] - 1 if tree_indptr.dim() else -1
    _need_i32(device, "tree_indptr", tree_indptr, bs + 1)
    if add_lens is not None:
        _need_i32(device, "add_lens", add_lens, bs)
    if seq_slots is not None:
        _need_i32(device, "seq_slots", seq_slots, bs)
    if lens_before is not None:
        _need_i32(device, "lens_before", lens_before, cache.max_seqs)
    if slots is None:
        slots = _empty(stream, num_tokens, dtype=torch.int64, device=cache.k_pages.device)
    elif slots.dtype is not torch.int64 or slots.shape != (num_tokens,) or not slots.is_contiguous() or slots.get_device() != device:
        raise CsgmvError(-1, f"slots must be a contiguous int64 tensor of shape ({num_tokens},) on cuda:{device}")
    if positions is None:
        positions = _empty(stream, num_tokens, dtype=torch.int32, device=cache.k_pages.device)
    else:
        _need_i32(device, "positions", positions, num_tokens)
    rc = lib().csgmv_kv_extend(cache._ref, _at(add_lens), tree_indptr.data_ptr(), _at(seq_slots), bs, num_tokens,
                               slots.data_ptr(), positions.data_ptr(), _at(lens_before), _raw_stream(stream, device))
    if rc:
        _check(rc)
    return slots, positions


def csgmv_kv_append(cache: KvCache, layer: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    positions: torch.Tensor | None = None, rope: Rope | None = None, q: torch.Tensor | None = None,
                    q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None) -> None:
    """Rows of k (turned by positions if there is a rope) and v (tokens,
    kv_heads, head_dim) into their slots of a layer of the cache, and q
    (tokens, heads, head_dim) turned into q_out (None: in place).  k_out, which
    may be k, gets the turned keys too."""
    n, d, dtype, device = k.shape[0], cache.head_dim, cache.dtype, cache.device
    ks = _head_strides("k", k, n, cache.num_kv_heads, d, dtype, device)
    vs = _head_strides("v", v, n, cache.num_kv_heads, d, dtype, device)
    if slots.dtype is not torch.int64 or slots.shape != (n,) or not slots.is_contiguous() or slots.get_device() != device:
        raise CsgmvError(-1, f"slots must be a contiguous int64 tensor of shape ({n},) on cuda:{device}")
    if rope is not None:
        if rope.head_dim != d or rope.device != device or positions is None:
            raise CsgmvError(-1, f"a rope for heads of {rope.head_dim} on cuda:{rope.device} and no or some positions, for heads "
                                 f"of {d} on cuda:{device}")
        _need_i32(device, "positions", positions, n)
    qs = qos = kos = (0, 0)
    hq = 0
    if q is not None:
        qs = _head_strides("q", q, n, None, d, dtype, device)
        hq = q.shape[1]
        if q_out is None or q_out is q:
            q_out, qos = q, qs
        else:
            qos = _head_strides("q_out", q_out, n, hq, d, dtype, device)
    elif q_out is not None:
        raise CsgmvError(-1, "q_out without q")
    if k_out is not None:
        kos = _head_strides("k_out", k_out, n, cache.num_kv_heads, d, dtype, device)
    rc = lib().csgmv_kv_append(
        cache._ref, layer, None if rope is None else rope._ref, _at(positions), slots.data_ptr(), n, _at(q), qs[0], qs[1], hq,
        k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], _at(q_out), qos[0], qos[1], _at(k_out), kos[0], kos[1],
        _raw_stream(stream, device))
    if rc:
        _check(rc)


class TokenCounts:
    """How often each of max_seqs sequences holds each token, empty at first.

      counts    int32 (max_seqs, vocab_size): times given, plus 2^30 if the prompt
                has it
      seen      int32 (max_seqs, vocab_size): its first num_seen[s] entries are the
                tokens that sequence s holds, in no certain order
      num_seen  int32 (max_seqs,)"""

    def __init__(self, max_seqs: int, vocab_size: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.counts = torch.zeros((max_seqs, vocab_size), **i32)
        self.seen = torch.zeros((max_seqs, vocab_size), **i32)
        self.num_seen = torch.zeros(max_seqs, **i32)
        self.status = torch.zeros(1, **i32)
        self.max_seqs, self.vocab_size, self.device = int(max_seqs), int(vocab_size), self.status.get_device()
        self.c = _TokenCountsC(self.counts.data_ptr(), self.seen.data_ptr(), self.num_seen.data_ptr(), self.status.data_ptr(),
                               max_seqs, vocab_size)
        self._ref = ctypes.byref(self.c)

    def device_status(self) -> int:
        return int(self.status.item())


def csgmv_count_tokens(counts: TokenCounts, tokens: torch.Tensor, tree_indptr: torch.Tensor,
                       accept_index: torch.Tensor | None = None, accept_len: torch.Tensor | None = None,
                       seq_slots: torch.Tensor | None = None, prompt: bool = False, stream=None) -> None:
    """Counts the tokens of request b's rows (its first accept_len[b], or its
    rows accept_index[b, j]) for its sequence; prompt: as its prompt."""
    device, bs = counts.device, tree_indptr.shape[0] - 1 if tree_indptr.dim() else -1
    n, width = tokens.numel(), 0
    _need_i32(device, "tokens", tokens, n)
    _need_i32(device, "tree_indptr", tree_indptr, bs + 1)
    if accept_index is not None:
        width = accept_index.shape[-1]
        _need_i32(device, "accept_index", accept_index, bs, width)
    if accept_len is not None:
        _need_i32(device, "accept_len", accept_len, bs)
    if seq_slots is not None:
        _need_i32(device, "seq_slots", seq_slots, bs)
    rc = lib().csgmv_count_tokens(counts._ref, tokens.data_ptr(), n, tree_indptr.data_ptr(), _at(accept_index), width,
                                  _at(accept_len), _at(seq_slots), bs, prompt, _raw_stream(stream, device))
    if rc:
        _check(rc)


def csgmv_count_reset(counts: TokenCounts, seqs: torch.Tensor, stream=None) -> None:
    """Empties sequences."""
    n = seqs.numel()
    _need_i32(counts.device, "seqs", seqs, n)
    _check(lib().csgmv_count_reset(counts._ref, seqs.data_ptr(), n, _raw_stream(stream, counts.device)))


def csgmv_count_fork(counts: TokenCounts, parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
    """Sequence children[i] becomes a copy of sequence parents[i]."""
    n = parents.numel()
    _need_i32(counts.device, "parents", parents, n)
    _need_i32(counts.device, "children", children, n)
    _check(lib().csgmv_count_fork(counts._ref, parents.data_ptr(), children.data_ptr(), n, _raw_stream(stream, counts.device)))


class LogitRules:
    """What csgmv_process_logits does to the rows of a batch of requests, over
    caller-owned tensors whose contents may change from call to call; each part
    may be None.

      counts       TokenCounts that the penalties go by (None: a row's own branch)
      repetition, frequency, presence, temperature   f32 (bs,)
      bias         (indptr int32 (bs + 1,), tokens int32 (total,), values f32
                   (total,)): entries of request b in increasing order of tokens
      allow        int32 (masks, words): bit v % 32 of word v / 32 lets token v through
      allow_index  int32 (rows,): each row's mask, or -1"""

    def __init__(self, counts: TokenCounts | None = None, repetition: torch.Tensor | None = None,
                 frequency: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                 temperature: torch.Tensor | None = None, bias: tuple | None = None, allow: torch.Tensor | None = None,
                 allow_index: torch.Tensor | None = None, device="cuda"):
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = at = self.status.get_device()
        _need(self.status.is_cuda, "the rules' device must be a CUDA device")
        _need(counts is None or counts.device == at, f"the counts are on another device than cuda:{at}")
        self.counts, self.bias, self.allow, self.allow_index = counts, bias, allow, allow_index
        self.repetition, self.frequency, self.presence, self.temperature = repetition, frequency, presence, temperature
        self.bs = None
        c = _LogitRulesC()
        if counts is not None:
            c.counts = ctypes.pointer(counts.c)
        for name in ("repetition", "frequency", "presence", "temperature"):
            t = getattr(self, name)
            if t is None:
                continue
            self.bs = t.shape[0] if self.bs is None and t.dim() else self.bs
            _need_f32(at, name, t, self.bs)
            _need(t.is_contiguous(), f"{name} must be contiguous")
            setattr(c, name, t.data_ptr())
        if bias is not None:
            indptr, tokens, values = bias
            total = tokens.numel()
            self.bs = indptr.shape[0] - 1 if self.bs is None and indptr.dim() else self.bs
            _need_i32(at, "bias indptr", indptr, self.bs + 1)
            _need_i32(at, "bias tokens", tokens, total)
            _need_f32(at, "bias values", values, total)
            _need(values.is_contiguous(), "bias values must be contiguous")
            c.bias_indptr, c.bias_tokens, c.bias_values, c.bias_total = indptr.data_ptr(), tokens.data_ptr(), values.data_ptr(), total
        self.rows = None
        _need((allow is None) == (allow_index is None), "allow and allow_index go together")
        if allow is not None:
            _need_i32(at, "allow", allow, None, None)
            _need_i32(at, "allow_index", allow_index, None)
            self.rows = allow_index.shape[0]
            c.allow, c.allow_index = allow.data_ptr(), allow_index.data_ptr()
            c.num_allow, c.allow_words = allow.shape
        c.status = self.status.data_ptr()
        self.c = c
        self._ref = ctypes.byref(c)

    def device_status(self) -> int:
        return int(self.status.item())


def csgmv_process_logits(logits: torch.Tensor, tree_indptr: torch.Tensor, rules: LogitRules, out: torch.Tensor | None = None,
                         draft_tokens: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                         seq_slots: torch.Tensor | None = None, softmax: bool = True, stream=None) -> torch.Tensor:
    """out (rows, vocab; f32, allocated on the call's stream unless given; may be
    logits): logits (rows, vocab; bf16, f16 or f32) of request b's rows after the
    rules, as probabilities, or as they are without softmax.  draft_tokens (int32,
    (rows,)) and mask (int32, (rows, words), of csgmv_build_draft_tree): the tokens
    of a row's own branch count as given."""
    device, dtype = rules.device, logits.dtype
    if len(logits.shape) != 2 or dtype not in _DTYPES or logits.get_device() != device or logits.shape[0] and logits.stride(1) != 1:
        raise CsgmvError(-1, f"logits must be (rows, vocab) of bf16, f16 or f32 on cuda:{device}, the rows dense")
    n, vocab = logits.shape
    bs = tree_indptr.shape[0] - 1 if tree_indptr.dim() else -1
    _need_i32(device, "tree_indptr", tree_indptr, bs + 1)
    if rules.bs is not None and rules.bs != bs or rules.rows is not None and rules.rows != n:
        raise CsgmvError(-1, f"rules for {rules.bs} requests and {rules.rows} rows, a batch of {bs} and {n}")
    if seq_slots is not None:
        _need_i32(device, "seq_slots", seq_slots, bs)
    words = 0
    if (mask is None) != (draft_tokens is None):
        raise CsgmvError(-1, "draft_tokens and mask go together")
    if mask is not None:
        words = mask.shape[-1]
        _need_i32(device, "mask", mask, n, words)
        _need_i32(device, "draft_tokens", draft_tokens, n)
    if out is None:
        out = _empty(stream, (n, vocab), dtype=torch.float32, device=logits.device)
    else:
        _need_f32(device, "out", out, n, vocab)
        if n and out.stride(1) != 1:
            raise CsgmvError(-1, "out must have dense rows")
    rc = lib().csgmv_process_logits(logits.data_ptr(), _DTYPES[dtype], logits.stride(0) if n > 1 else vocab, tree_indptr.data_ptr(),
                                    _at(seq_slots), bs, n, vocab, rules._ref, _at(draft_tokens), _at(mask), words, softmax,
                                    out.data_ptr(), out.stride(0) if n > 1 else vocab, _raw_stream(stream, device))
    if rc:
        _check(rc)
    return out
