"""ctypes binding of libcsgmv.so (include/csgmv.h), same names as the C ABI.

Argument marshalling only: torch supplies device memory and the current CUDA
stream, every step of the path runs in the library's kernels.  There is no
fallback: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
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
    1: "BAD_SEQ", 2: "BAD_PAGE", 4: "CAPACITY", 8: "BAD_LENS", 16: "BAD_TREE", 32: "BAD_TOKEN", 1 << 30: "TIMEOUT",
}

EXPORTED = ["csgmv_last_error", "csgmv_version", "csgmv_chunk_size", "csgmv_batch_info_capacity",
            "csgmv_build_batch_info", "csgmv_build_lm_head_batch_info", "csgmv_shrink", "csgmv_expand", "csgmv_qkv", "csgmv_qkv_workspace_bytes",
            "csgmv_qkv_static_scratch", "embedding_lora_a", "embedding_lora_a_extra", "extra_token_embedding",
            "csgmv_expand_sliced", "csgmv_qkv_sliced", "csgmv_qkv_path", "csgmv_tile_table_ints",
            "embedding_lora_a_transposed", "csgmv_transpose_embedding",
            "csgmv_kv_scratch_ints", "csgmv_kv_commit", "csgmv_kv_fork", "csgmv_kv_free", "csgmv_kv_compact",
            "csgmv_kv_copy_pages", "csgmv_tree_attention", "csgmv_tree_attention_workspace_bytes",
            "csgmv_build_draft_tree", "csgmv_verify_drafts"]

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
