"""Thin Python binding of the C ABI in ``include/pkv.h`` (argument marshalling only).

Every step of the decode path runs in the CUDA kernels of ``libpkv.so``; this
module only turns tensors into pointers and sizes, passes the current CUDA
stream, and raises on a negative status.  There is no CPU fallback: if the
library is missing the import fails.

Function names follow the C entry points without their ``pkv_`` prefix.
PyTorch provides device memory and streams.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_180_gb300.build` "
                      "(the CUDA path has no fallback)")

_lib = ctypes.CDLL(LIB_PATH)

PKV_OK = 0
DEV_BAD_SLOT = 1
DEV_BAD_CONTEXT = 2
DEV_BAD_PAGE = 4
DEV_TIMEOUT = 8
DEV_BAD_PATH = 16


class PkvPool(ctypes.Structure):
    """Mirror of ``pkv_pool``."""
    _fields_ = [("k_base", ctypes.c_void_p), ("v_base", ctypes.c_void_p), ("page_stride_bytes", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class PkvStepPlan(ctypes.Structure):
    """Mirror of ``pkv_step_plan``."""
    _fields_ = [("num_finished", ctypes.c_int32), ("finished_request", ctypes.POINTER(ctypes.c_int64)),
                ("num_admitted", ctypes.c_int32), ("admitted_request", ctypes.POINTER(ctypes.c_int64)),
                ("admitted_slot", ctypes.POINTER(ctypes.c_int32)),
                ("num_appends", ctypes.c_int32), ("append_request", ctypes.POINTER(ctypes.c_int64)),
                ("append_position", ctypes.POINTER(ctypes.c_int32)),
                ("append_slot_mapping", ctypes.POINTER(ctypes.c_int32)),
                ("num_decode", ctypes.c_int32), ("decode_slot", ctypes.POINTER(ctypes.c_int32)),
                ("context_lens", ctypes.POINTER(ctypes.c_int32)), ("block_tables", ctypes.POINTER(ctypes.c_int32)),
                ("max_blocks", ctypes.c_int32)]


class PkvSchedStats(ctypes.Structure):
    """Mirror of ``pkv_sched_stats``."""
    _fields_ = [("pool_pages", ctypes.c_int32), ("peak_active", ctypes.c_int32), ("largest_batch", ctypes.c_int32),
                ("peak_pages", ctypes.c_int32), ("admission_waits", ctypes.c_int32), ("free_pages", ctypes.c_int32),
                ("credits_in_use", ctypes.c_int32), ("active", ctypes.c_int32), ("queued", ctypes.c_int32),
                ("steps", ctypes.c_int64)]


_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_PP = ctypes.POINTER(PkvPool)

EXPORTS = {
    # name: (restype, argtypes)
    "pkv_kv_pool_bytes": (_Z, [_I, _I, _I, _I]),
    "pkv_kv_pool_create": (_I, [_P, _P, _L, _I, _I, _I, _I, _PP]),
    "pkv_kv_append": (_I, [_PP, _P, _P, _P, _I, _P, _P]),
    "pkv_decode_workspace_bytes": (_Z, [_I, _I, _I]),
    "pkv_paged_decode_attention": (_I, [_PP, _P, _P, _I, _P, _L, _P, _I, _I, _F, _P, _Z, _P, _P]),
    "pkv_paged_decode_attention_ctas": (_I, [_PP, _P, _P, _I, _P, _L, _P, _I, _I, _F, _P, _Z, _P, _I, _P]),
    "pkv_decode_max_ctas": (_I, []),
    "pkv_decode_plan": (_I, [_I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "pkv_status_string": (ctypes.c_char_p, [_I]),
    "pkv_paged_decode_attention_noalloc": (_I, [_PP, _P, _P, _I, _P, _L, _P, _I, _I, _F, _P, _P]),
    "pkv_decode_step": (_I, [_PP, _P, _P, _P, _P, _P, _I, _P, _L, _P, _I, _I, _F, _P, _Z, _P, _P]),
    "pkv_decode_step_ex": (_I, [_PP, _P, _P, _P, _P, _P, _I, _P, _L, _P, _I, _I, _F, _P, _Z, _P, ctypes.c_uint, _P]),
    "pkv_paged_prefill_attention": (_I, [_PP, _P, _P, _I, _I, _P, _P, _L, _P, _I, _I, _I, _F, _P, _P]),
    "pkv_paged_prefill_attention_ex": (_I, [_PP, _P, _P, _I, _I, _P, _P, _L, _P, _I, _I, _I, _F, _P, ctypes.c_uint,
                                            _P]),
    "pkv_paged_tree_attention": (_I, [_PP, _P, _P, _I, _I, _P, _P, _L, _P, _L, _P, _I, _I, _I, _F, _P, _Z, _P,
                                      ctypes.c_uint, _P]),
    "pkv_tree_workspace_bytes": (_Z, [_I, _I, _I, _I]),
    "pkv_tree_commit": (_I, [_PP, _P, _L, _L, _I, _P, _P, _P, _L, _P, _I, _I, _I, _P, _P, _P]),
    "pkv_kv_copy_pages": (_I, [_PP, _P, _P, _I, _P, _P]),
    "pkv_alloc_create": (_I, [_I, _I, _I, _I, _I, _P, ctypes.POINTER(_P)]),
    "pkv_alloc_destroy": (None, [_P]),
    "pkv_alloc_admit": (_I, [_P, _I, _I, _I, ctypes.POINTER(ctypes.c_int32)]),
    "pkv_alloc_page": (_I, [_P, _I, _I, _I, ctypes.POINTER(ctypes.c_int32)]),
    "pkv_alloc_free_seq": (_I, [_P, _I]),
    "pkv_alloc_block_tables": (ctypes.POINTER(ctypes.c_int32), [_P]),
    "pkv_alloc_state": (_I, [_P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]),
    "pkv_alloc_fork": (_I, [_P, _I, _I, _I, _I, _P, _P, _I, ctypes.POINTER(ctypes.c_int32)]),
    "pkv_alloc_write_page": (_I, [_P, _I, _I, _I, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]),
    "pkv_alloc_truncate": (_I, [_P, _I, _I]),
    "pkv_alloc_compact": (_I, [_P, _P, _P, _I, ctypes.POINTER(ctypes.c_int32)]),
    "pkv_alloc_page_refs": (_I, [_P, _I]),
    "pkv_sched_create": (_I, [_I, _I, _I, _I, _I, _P, ctypes.POINTER(_P)]),
    "pkv_sched_destroy": (None, [_P]),
    "pkv_sched_submit": (_I, [_P, _L, _I, _I]),
    "pkv_sched_step": (_I, [_P, ctypes.POINTER(PkvStepPlan)]),
    "pkv_sched_stats_get": (_I, [_P, ctypes.POINTER(PkvSchedStats)]),
}

NOALLOC_MAX_SEQS = 512  # PKV_NOALLOC_MAX_SEQS
OVERLAP_PREVIOUS = 1  # PKV_OVERLAP_PREVIOUS
OUT_BF16 = 2  # PKV_OUT_BF16

for _name, (_res, _args) in EXPORTS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class PkvError(RuntimeError):
    def __init__(self, where: str, code: int):
        super().__init__(f"{where}: {status_string(code)} ({code})")
        self.code = code


def _check(where: str, rc: int) -> None:
    if rc != PKV_OK:
        raise PkvError(where, rc)


def status_string(code: int) -> str:
    return _lib.pkv_status_string(int(code)).decode()


# The current stream's handle and the current device without the Stream object that
# torch.cuda.current_stream() builds (2.9 us a call on the Grace host, against 0.2 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_cuda_ready = False


def _stream(stream) -> int:
    global _cuda_ready
    if stream is not None:
        return int(stream.cuda_stream)
    if _cuda_ready:
        return _raw_stream(_current_device())
    _cuda_ready = _raw_stream is not None and torch.cuda.is_initialized()
    return int(torch.cuda.current_stream().cuda_stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else int(t.data_ptr())


# ---------------------------------------------------------------------------
def kv_pool_bytes(num_pages: int, page_tokens: int = 16, num_kv_heads: int = 8, head_dim: int = 64) -> int:
    return int(_lib.pkv_kv_pool_bytes(num_pages, page_tokens, num_kv_heads, head_dim))


def kv_pool_create(k_pool: torch.Tensor | int, v_pool: torch.Tensor | int, page_stride_bytes: int, num_pages: int,
                   page_tokens: int = 16, num_kv_heads: int = 8, head_dim: int = 64) -> PkvPool:
    """Descriptor for caller-owned pool memory (tensors or raw device addresses)."""
    kp = k_pool if isinstance(k_pool, int) else _ptr(k_pool)
    vp = v_pool if isinstance(v_pool, int) else _ptr(v_pool)
    desc = PkvPool()
    _check("pkv_kv_pool_create", _lib.pkv_kv_pool_create(kp, vp, page_stride_bytes, num_pages, page_tokens,
                                                         num_kv_heads, head_dim, ctypes.byref(desc)))
    return desc


class KVPool:
    """One interleaved pool buffer ([page][K|V][kv_head][row][dim] bf16) owned by a torch tensor."""

    def __init__(self, num_pages: int, page_tokens: int = 16, num_kv_heads: int = 8, head_dim: int = 64,
                 device="cuda", buffer: torch.Tensor | None = None):
        nbytes = kv_pool_bytes(num_pages, page_tokens, num_kv_heads, head_dim)
        if buffer is None:
            buffer = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=device)
        assert buffer.numel() * buffer.element_size() >= nbytes
        self.buffer = buffer
        self.num_pages, self.page_tokens = num_pages, page_tokens
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        half = num_kv_heads * page_tokens * head_dim * 2
        base = _ptr(buffer)
        self.desc = kv_pool_create(base, base + half, 2 * half, num_pages, page_tokens, num_kv_heads, head_dim)

    def view(self) -> torch.Tensor:
        """The pool as [num_pages, 2, num_kv_heads, page_tokens, head_dim] bf16."""
        return self.buffer[: self.num_pages * 2 * self.num_kv_heads * self.page_tokens * self.head_dim].view(
            self.num_pages, 2, self.num_kv_heads, self.page_tokens, self.head_dim)


def kv_append(pool: KVPool | PkvPool, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
              status: torch.Tensor | None = None, stream=None) -> None:
    desc = pool.desc if isinstance(pool, KVPool) else pool
    n = int(slot_mapping.shape[0])
    _check("pkv_kv_append", _lib.pkv_kv_append(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                               n, _ptr(status), _stream(stream)))


def decode_workspace_bytes(num_seqs: int, num_q_heads: int = 32, head_dim: int = 64) -> int:
    return int(_lib.pkv_decode_workspace_bytes(num_seqs, num_q_heads, head_dim))


def decode_workspace(num_seqs: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for pkv_paged_decode_attention (zeroed once; calls keep it valid)."""
    return torch.zeros(decode_workspace_bytes(num_seqs), dtype=torch.uint8, device=device)


def decode_max_ctas() -> int:
    return int(_lib.pkv_decode_max_ctas())


def decode_plan(num_seqs: int, max_context: int) -> tuple[int, int]:
    g, n = _I(0), _I(0)
    _check("pkv_decode_plan", _lib.pkv_decode_plan(num_seqs, max_context, ctypes.byref(g), ctypes.byref(n)))
    return g.value, n.value


def paged_decode_attention(pool: KVPool | PkvPool, out: torch.Tensor, q: torch.Tensor, block_tables: torch.Tensor,
                           block_table_stride: int, context_lens: torch.Tensor, max_context: int, scale: float,
                           workspace: torch.Tensor, status: torch.Tensor | None = None, num_ctas: int = 0,
                           stream=None) -> None:
    """out[s, h, :] = softmax(scale * q[s, h] . K[h // group]) V over the cached tokens of sequence s."""
    desc = pool.desc if isinstance(pool, KVPool) else pool
    num_seqs, num_q_heads = int(q.shape[0]), int(q.shape[1])
    ws_bytes = workspace.numel() * workspace.element_size()
    if num_ctas:
        rc = _lib.pkv_paged_decode_attention_ctas(ctypes.byref(desc), _ptr(out), _ptr(q), num_q_heads,
                                                  _ptr(block_tables), block_table_stride, _ptr(context_lens),
                                                  num_seqs, max_context, scale, _ptr(workspace), ws_bytes,
                                                  _ptr(status), num_ctas, _stream(stream))
    else:
        rc = _lib.pkv_paged_decode_attention(ctypes.byref(desc), _ptr(out), _ptr(q), num_q_heads,
                                             _ptr(block_tables), block_table_stride, _ptr(context_lens),
                                             num_seqs, max_context, scale, _ptr(workspace), ws_bytes,
                                             _ptr(status), _stream(stream))
    _check("pkv_paged_decode_attention", rc)


def decode_step(pool: KVPool | PkvPool, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                out: torch.Tensor, q: torch.Tensor, block_tables: torch.Tensor, block_table_stride: int,
                context_lens: torch.Tensor, max_context: int, scale: float, workspace: torch.Tensor,
                status: torch.Tensor | None = None, stream=None, overlap_previous: bool = False) -> None:
    """kv_append of one new token per sequence (position context_lens[s] - 1) fused with
    paged_decode_attention, in one launch.  overlap_previous: launch with programmatic stream
    serialization (PKV_OVERLAP_PREVIOUS; only when the kernel before it on the stream writes
    none of the lengths, tables or pool pages this step reads)."""
    desc = pool.desc if isinstance(pool, KVPool) else pool
    num_seqs, num_q_heads = int(q.shape[0]), int(q.shape[1])
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = _lib.pkv_decode_step_ex(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(out),
                                 _ptr(q), num_q_heads, _ptr(block_tables), block_table_stride, _ptr(context_lens),
                                 num_seqs, max_context, scale, _ptr(workspace), ws_bytes, _ptr(status),
                                 OVERLAP_PREVIOUS if overlap_previous else 0, _stream(stream))
    _check("pkv_decode_step_ex", rc)


def paged_prefill_attention(pool: KVPool | PkvPool, out: torch.Tensor, q: torch.Tensor, query_start: torch.Tensor,
                            block_tables: torch.Tensor, block_table_stride: int, context_lens: torch.Tensor,
                            max_query: int, max_context: int, scale: float, status: torch.Tensor | None = None,
                            stream=None, overlap_previous: bool = False) -> None:
    """Causal attention of the last n_s cached tokens of each sequence (rows query_start[s] ..).
    overlap_previous: launch with PKV_OVERLAP_PREVIOUS (only when the kernel before it on the
    stream writes none of q, query_start, context_lens or block_tables, e.g. the prompt's
    kv_append)."""
    desc = pool.desc if isinstance(pool, KVPool) else pool
    num_seqs = int(context_lens.shape[0])
    rows = min(int(q.shape[0]), int(out.shape[0]))
    rc = _lib.pkv_paged_prefill_attention_ex(ctypes.byref(desc), _ptr(out), _ptr(q), int(q.shape[1]), rows,
                                             _ptr(query_start), _ptr(block_tables), block_table_stride,
                                             _ptr(context_lens), num_seqs, max_query, max_context, scale, _ptr(status),
                                             OVERLAP_PREVIOUS if overlap_previous else 0, _stream(stream))
    _check("pkv_paged_prefill_attention_ex", rc)


def paged_decode_attention_noalloc(pool: KVPool | PkvPool, out: torch.Tensor, q: torch.Tensor,
                                   block_tables: torch.Tensor, block_table_stride: int, context_lens: torch.Tensor,
                                   max_context: int, scale: float, status: torch.Tensor | None = None,
                                   stream=None) -> None:
    """paged_decode_attention without a workspace, for callers that cannot allocate device memory.

    The library keeps the split-context partial states in one fixed device array (up to
    NOALLOC_MAX_SEQS sequences) shared by every call on a device: calls must not overlap on the
    GPU, and the first call on a device should come before any stream capture there.
    """
    desc = pool.desc if isinstance(pool, KVPool) else pool
    num_seqs, num_q_heads = int(q.shape[0]), int(q.shape[1])
    rc = _lib.pkv_paged_decode_attention_noalloc(ctypes.byref(desc), _ptr(out), _ptr(q), num_q_heads,
                                                 _ptr(block_tables), block_table_stride, _ptr(context_lens),
                                                 num_seqs, max_context, scale, _ptr(status), _stream(stream))
    _check("pkv_paged_decode_attention_noalloc", rc)


def _refuse(where: str, t: torch.Tensor, dtype) -> None:
    raise ValueError(f"{where}: expected a contiguous {dtype} tensor on the current device (cuda:{_current_device()}), got "
                     f"{t.dtype} on {t.device} with strides {tuple(t.stride())}")


def _status_ptr(where: str, status: torch.Tensor | None, dev: int) -> int | None:
    if status is None:
        return None
    if (status.dtype is not _I32 and status.dtype is not torch.uint32) or status.get_device() != dev or status.numel() < 1:
        raise ValueError(f"{where}: status is an int32 word on the current device (cuda:{dev}), got {status.numel()} of "
                         f"{status.dtype} on {status.device}")
    return status.data_ptr()


def tree_workspace_bytes(num_seqs: int, max_query: int, num_q_heads: int = 32, head_dim: int = 64) -> int:
    return int(_lib.pkv_tree_workspace_bytes(num_seqs, max_query, num_q_heads, head_dim))


def tree_workspace(num_seqs: int, max_query: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for pkv_paged_tree_attention (zeroed once; calls keep it valid)."""
    return torch.zeros(tree_workspace_bytes(num_seqs, max_query), dtype=torch.uint8, device=device)


def paged_tree_attention(pool: KVPool | PkvPool, out: torch.Tensor, q: torch.Tensor, query_start: torch.Tensor,
                         tree_mask: torch.Tensor, block_tables: torch.Tensor, block_table_stride: int,
                         context_lens: torch.Tensor, max_query: int, max_context: int, scale: float,
                         workspace: torch.Tensor, status: torch.Tensor | None = None, stream=None,
                         overlap_previous: bool = False) -> None:
    """Attention of the last n_s cached tokens of each sequence, the nodes of a tree: every node attends
    to the prefix before them and to the nodes whose bits its row of tree_mask (int32 [rows, words]) has.
    out: float32 or bfloat16 [rows, heads, dim].  overlap_previous: launch with PKV_OVERLAP_PREVIOUS (only
    when the kernel before it on the stream writes none of q, query_start, context_lens or block_tables,
    e.g. the drafted tokens' kv_append)."""
    where = "pkv_paged_tree_attention"
    # the kernel sees pointers only: type, order and device have to be what it takes them for
    dev, kind = _current_device(), out.dtype
    for t in (query_start, tree_mask, context_lens):
        if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous():
            _refuse(where, t, _I32)
    if q.dtype is not _BF16 or q.get_device() != dev or not q.is_contiguous():
        _refuse(where, q, _BF16)
    if block_tables.dtype is not _I32 or block_tables.get_device() != dev or block_tables.stride(-1) != 1:
        _refuse(where, block_tables, _I32)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(where, workspace, "uint8")
    if (kind is not _F32 and kind is not _BF16) or out.get_device() != dev or not out.is_contiguous():
        _refuse(where, out, "float32 or bfloat16")
    num_seqs, shape, out_shape, mask_shape = context_lens.numel(), q.shape, out.shape, tree_mask.shape
    if len(shape) != 3 or out_shape[1:] != shape[1:] or len(mask_shape) != 2 or query_start.numel() != num_seqs + 1:
        raise ValueError(f"{where}: q and out are [rows, heads, dim], tree_mask [rows, words], query_start [seqs + 1]")
    flags = (OVERLAP_PREVIOUS if overlap_previous else 0) | (OUT_BF16 if kind is _BF16 else 0)
    rc = _lib.pkv_paged_tree_attention(
        ctypes.byref(pool.desc if isinstance(pool, KVPool) else pool), out.data_ptr(), q.data_ptr(), shape[1],
        min(shape[0], out_shape[0], mask_shape[0]), query_start.data_ptr(), tree_mask.data_ptr(), mask_shape[1],
        block_tables.data_ptr(), block_table_stride, context_lens.data_ptr(), num_seqs, max_query, max_context, scale,
        workspace.data_ptr(), workspace.nbytes, _status_ptr(where, status, dev), flags, _stream(stream))
    if rc:
        raise PkvError(where, rc)


def tree_commit(pool: KVPool | PkvPool, block_tables: torch.Tensor, block_table_stride: int, layer_stride: int,
                num_layers: int, query_start: torch.Tensor, context_lens: torch.Tensor, accepted: torch.Tensor,
                accept_counts: torch.Tensor, max_context: int, new_context_lens: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> None:
    """Move the rows of each sequence's accepted path (accepted: int32 [seqs, width], ascending nodes, the
    first accept_counts[s] of row s) behind its committed prefix in every layer; new_context_lens receives
    the lengths after it."""
    where = "pkv_tree_commit"
    dev = _current_device()
    for t in (query_start, context_lens, accepted, accept_counts):
        if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous():
            _refuse(where, t, _I32)
    if block_tables.dtype is not _I32 or block_tables.get_device() != dev or block_tables.stride(-1) != 1:
        _refuse(where, block_tables, _I32)
    num_seqs, shape = context_lens.numel(), accepted.shape
    if len(shape) != 2 or shape[0] != num_seqs or accept_counts.numel() != num_seqs or \
            query_start.numel() != num_seqs + 1:
        raise ValueError(f"{where}: accepted is [seqs, width], accept_counts [seqs], query_start [seqs + 1]")
    new = None
    if new_context_lens is not None:
        new = new_context_lens.data_ptr()
        if new_context_lens.dtype is not _I32 or new_context_lens.get_device() != dev or \
                not new_context_lens.is_contiguous():
            _refuse(where, new_context_lens, _I32)
        if new_context_lens.numel() < num_seqs:
            raise ValueError(f"{where}: new_context_lens has {new_context_lens.numel()} entries for {num_seqs} sequences")
    width = shape[1]
    rc = _lib.pkv_tree_commit(
        ctypes.byref(pool.desc if isinstance(pool, KVPool) else pool), block_tables.data_ptr(), block_table_stride,
        layer_stride, num_layers, query_start.data_ptr(), context_lens.data_ptr(), accepted.data_ptr(), width,
        accept_counts.data_ptr(), num_seqs, width, max_context, new, _status_ptr(where, status, dev), _stream(stream))
    if rc:
        raise PkvError(where, rc)


def kv_copy_pages(pool: KVPool | PkvPool, src_pages: torch.Tensor, dst_pages: torch.Tensor,
                  status: torch.Tensor | None = None, stream=None) -> None:
    """Copy page src_pages[i] onto page dst_pages[i] (int32; a negative id is padding), K and V."""
    where = "pkv_kv_copy_pages"
    n, dev = src_pages.numel(), _current_device()
    for t in (src_pages, dst_pages):
        if t.dtype is not _I32 or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"{where}: page ids are contiguous int32 tensors, as many sources as destinations")
        if t.get_device() != dev and not (n == 0 or t.get_device() == -1 and t.is_pinned()):
            raise ValueError(f"{where}: page ids on {t.device}; they lie on the current device (cuda:{dev}) or in pinned "
                             "host memory")
    rc = _lib.pkv_kv_copy_pages(ctypes.byref(pool.desc if isinstance(pool, KVPool) else pool), src_pages.data_ptr(),
                                dst_pages.data_ptr(), n, _status_ptr(where, status, dev), _stream(stream))
    if rc:
        raise PkvError(where, rc)


class Allocator:
    """Host page allocator of ``libpkv.so`` (see ``pkv_alloc_*``): admission credits, lazy pages
    from a LIFO free list, release of a sequence's pages.  Methods raise PkvError on a negative
    status, except ``admit``, which returns the status (PKV_OK, NO_CREDIT or EXCEEDS_POOL)."""

    OK, NO_CREDIT, EXCEEDS_POOL = 0, -13, -9

    def __init__(self, num_pages: int, num_layers: int = 1, page_tokens: int = 16, max_context: int = 2048,
                 max_seqs: int = 32, free_order=None):
        import numpy as np
        self._np = np
        self.num_pages, self.num_layers, self.max_seqs = num_pages, num_layers, max_seqs
        self.max_blocks = -(-max_context // page_tokens)
        order = None
        if free_order is not None:
            self._order = np.ascontiguousarray(free_order, dtype=np.int32)
            order = self._order.ctypes.data
        h = ctypes.c_void_p()
        _check("pkv_alloc_create", _lib.pkv_alloc_create(num_pages, num_layers, page_tokens, max_context, max_seqs,
                                                         order, ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _lib.pkv_alloc_destroy(h)
            self._h = None

    def admit(self, seq: int, prompt_tokens: int, max_new_tokens: int) -> tuple[int, int]:
        """(status, credits) of admitting a request into ``seq``."""
        c = ctypes.c_int32(0)
        rc = _lib.pkv_alloc_admit(self._h, seq, prompt_tokens, max_new_tokens, ctypes.byref(c))
        if rc not in (self.OK, self.NO_CREDIT, self.EXCEEDS_POOL):
            raise PkvError("pkv_alloc_admit", rc)
        return rc, c.value

    def page(self, seq: int, layer: int, block: int) -> int:
        p = ctypes.c_int32(-1)
        _check("pkv_alloc_page", _lib.pkv_alloc_page(self._h, seq, layer, block, ctypes.byref(p)))
        return p.value

    def free_seq(self, seq: int) -> None:
        _check("pkv_alloc_free_seq", _lib.pkv_alloc_free_seq(self._h, seq))

    def fork(self, src_seq: int, dst_seq: int, tokens: int, max_new_tokens: int):
        """(status, source pages, new pages): dst_seq shares the first ``tokens`` tokens of src_seq; copy the
        pages (``kv_copy_pages``) before using the fork.  Status as for ``admit``."""
        np = self._np
        src, dst, n = np.zeros(self.num_layers, np.int32), np.zeros(self.num_layers, np.int32), ctypes.c_int32(0)
        rc = _lib.pkv_alloc_fork(self._h, src_seq, dst_seq, tokens, max_new_tokens, src.ctypes.data, dst.ctypes.data,
                                 self.num_layers, ctypes.byref(n))
        if rc not in (self.OK, self.NO_CREDIT, self.EXCEEDS_POOL):
            raise PkvError("pkv_alloc_fork", rc)
        k = n.value if rc == self.OK else 0
        return rc, src[:k].copy(), dst[:k].copy()

    def write_page(self, seq: int, layer: int, block: int) -> tuple[int, int]:
        """(page, shared page to copy into it first, or -1) of a block about to be written."""
        p, c = ctypes.c_int32(-1), ctypes.c_int32(-1)
        _check("pkv_alloc_write_page", _lib.pkv_alloc_write_page(self._h, seq, layer, block, ctypes.byref(p),
                                                                 ctypes.byref(c)))
        return p.value, c.value

    def truncate(self, seq: int, tokens: int) -> None:
        """Give back the pages behind the first ``tokens`` tokens."""
        _check("pkv_alloc_truncate", _lib.pkv_alloc_truncate(self._h, seq, tokens))

    def compact(self):
        """(source pages, destination pages) of the moves that put the used pages at 0 .. used - 1."""
        np = self._np
        src, dst = np.zeros(self.num_pages, np.int32), np.zeros(self.num_pages, np.int32)
        n = ctypes.c_int32(0)
        _check("pkv_alloc_compact", _lib.pkv_alloc_compact(self._h, src.ctypes.data, dst.ctypes.data, self.num_pages,
                                                           ctypes.byref(n)))
        return src[:n.value].copy(), dst[:n.value].copy()

    def page_refs(self, page: int) -> int:
        return int(_lib.pkv_alloc_page_refs(self._h, page))

    def block_tables(self):
        """A copy of the block table [max_seqs, num_layers, max_blocks]."""
        n = self.max_seqs * self.num_layers * self.max_blocks
        ptr = _lib.pkv_alloc_block_tables(self._h)
        return self._np.ctypeslib.as_array(ptr, shape=(n,)).copy().reshape(self.max_seqs, self.num_layers,
                                                                           self.max_blocks)

    def state(self) -> tuple[int, int]:
        """(free pages, credits in use)."""
        f, c = ctypes.c_int32(0), ctypes.c_int32(0)
        _check("pkv_alloc_state", _lib.pkv_alloc_state(self._h, ctypes.byref(f), ctypes.byref(c)))
        return f.value, c.value


class Scheduler:
    """Host page allocator + continuous-batching scheduler of ``libpkv.so`` (see ``pkv_sched_*``)."""

    def __init__(self, num_pages: int, num_layers: int = 1, page_tokens: int = 16, max_context: int = 2048,
                 num_slots: int = 32, free_order=None):
        import numpy as np
        self._np = np
        self.num_layers, self.num_slots = num_layers, num_slots
        order = None
        if free_order is not None:
            self._order = np.ascontiguousarray(free_order, dtype=np.int32)
            order = self._order.ctypes.data
        h = ctypes.c_void_p()
        _check("pkv_sched_create", _lib.pkv_sched_create(num_pages, num_layers, page_tokens, max_context, num_slots,
                                                         order, ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _lib.pkv_sched_destroy(h)
            self._h = None

    def submit(self, request_id: int, prompt_tokens: int, max_new_tokens: int) -> None:
        _check("pkv_sched_submit", _lib.pkv_sched_submit(self._h, int(request_id), int(prompt_tokens),
                                                         int(max_new_tokens)))

    def step(self) -> dict:
        """One step; returns copies of the plan as numpy arrays."""
        np = self._np
        plan = PkvStepPlan()
        _check("pkv_sched_step", _lib.pkv_sched_step(self._h, ctypes.byref(plan)))

        def arr(ptr, n, dt):
            if n == 0:
                return np.zeros(0, dtype=dt)
            return np.ctypeslib.as_array(ptr, shape=(n,)).astype(dt, copy=True)

        na, L, S = plan.num_appends, self.num_layers, self.num_slots
        return {
            "finished": arr(plan.finished_request, plan.num_finished, np.int64),
            "admitted": arr(plan.admitted_request, plan.num_admitted, np.int64),
            "admitted_slot": arr(plan.admitted_slot, plan.num_admitted, np.int32),
            "append_request": arr(plan.append_request, na, np.int64),
            "append_position": arr(plan.append_position, na, np.int32),
            "append_slot_mapping": arr(plan.append_slot_mapping, na * L, np.int32).reshape(L, na),
            "decode_slot": arr(plan.decode_slot, plan.num_decode, np.int32),
            "context_lens": arr(plan.context_lens, S, np.int32),
            "block_tables": arr(plan.block_tables, S * L * plan.max_blocks, np.int32).reshape(S, L, plan.max_blocks),
        }

    def stats(self) -> dict:
        st = PkvSchedStats()
        _check("pkv_sched_stats_get", _lib.pkv_sched_stats_get(self._h, ctypes.byref(st)))
        return {name: int(getattr(st, name)) for name, _ in PkvSchedStats._fields_}
