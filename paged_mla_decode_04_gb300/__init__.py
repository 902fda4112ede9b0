"""Paged MLA decode for GB300: thin Python binding of libmla_decode.so.

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch supplies device memory and streams. If the library is missing or
cannot be loaded this module raises; there is no fallback path.

Calls (same names as the C ABI in include/mla_decode.h):
  kv_write(pool, layer, new_rows, slot_mapping, workspace=None)
  workspace_size(batch, num_heads) / num_clusters()
  plan(context_lens, num_heads, page_size, window, workspace, num_clusters=0)
  decode(pool, layer, q, context_lens, softmax_scale, workspace, out,
         block_table=None | page_indptr + page_ids, window=0, lse=None)
  workspace_size_q / plan_q / decode_q: several query positions per request
  (q [batch, q_len, heads, 576]; causal within the step)
  uv_project(attn_out, w_uv, y, workspace=None)
  extend_tables / rope_write / prefill: a step of ragged chunks of new tokens
  (page tables from lengths, rotary latent write, 192/128 attention)
  get_error(workspace, clear=False)
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")

MLA_OK = 0
ERRORS = {-1: "MLA_ERR_ARG", -2: "MLA_ERR_UNSUPPORTED", -3: "MLA_ERR_WORKSPACE", -4: "MLA_ERR_CUDA"}
STATUS_BAD_PAGE = 0x1
STATUS_BAD_SLOT = 0x2
STATUS_PLAN_MISMATCH = 0x4
STATUS_TIMEOUT = 0x8
STATUS_BAD_LENGTH = 0x10
STATUS_NO_PAGES = 0x20
STATUS_BAD_POSITION = 0x40
DTYPE_BF16 = 0
DTYPE_FP8_E4M3 = 1
LATENT_DIM = 576
KV_LORA_RANK = 512
V_HEAD_DIM = 128
NOPE_DIM = 128
ROPE_DIM = 64
QK_HEAD_DIM = 192

EXPORTED = ["mla_kv_write", "mla_decode_workspace_size", "mla_decode_num_clusters",
            "mla_decode_plan", "mla_decode", "mla_uv_project", "mla_get_error",
            "mla_decode_noalloc", "mla_decode_workspace_size_q", "mla_decode_plan_q",
            "mla_decode_q", "mla_selftest_bounded_wait", "mla_extend_tables", "mla_rope_write",
            "mla_prefill", "mla_prefill_workspace_size"]
NOALLOC_SCRATCH_BYTES = 48 << 20


class MlaError(RuntimeError):
    pass


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_layers", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int), ("kv_scale", ctypes.c_float)]


_pack_pool = struct.Struct("@Piiiif0P").pack  # _Pool, its tail padding included
assert len(_pack_pool(0, 0, 0, 0, 0, 0.0)) == ctypes.sizeof(_Pool)

_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmla_decode.so (raises if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise MlaError("libmla_decode.so not built; run paged_mla_decode_04_gb300._build.build()")
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.mla_kv_write.argtypes = [ctypes.POINTER(_Pool), I, P, P, I, P, P]
    lib.mla_kv_write.restype = I
    lib.mla_decode_workspace_size.argtypes = [I, I]
    lib.mla_decode_workspace_size.restype = Z
    lib.mla_decode_num_clusters.argtypes = []
    lib.mla_decode_num_clusters.restype = I
    lib.mla_decode_plan.argtypes = [P, I, I, I, I, I, P, Z, P]
    lib.mla_decode_plan.restype = I
    lib.mla_decode.argtypes = [ctypes.POINTER(_Pool), I, P, P, P, I, P, I, I, ctypes.c_float, I,
                               P, P, P, P]
    lib.mla_decode.restype = I
    lib.mla_uv_project.argtypes = [P, P, P, I, I, P, P]
    lib.mla_uv_project.restype = I
    lib.mla_get_error.argtypes = [P, ctypes.POINTER(I), I, P]
    lib.mla_get_error.restype = I
    lib.mla_selftest_bounded_wait.argtypes = [I, ctypes.c_uint, P, P]
    lib.mla_selftest_bounded_wait.restype = I
    lib.mla_decode_noalloc.argtypes = [ctypes.POINTER(_Pool), I, P, P, P, I, P, I, I, ctypes.c_float,
                                       I, I, P, P, P, P]
    lib.mla_decode_noalloc.restype = I
    lib.mla_decode_workspace_size_q.argtypes = [I, I, I]
    lib.mla_decode_workspace_size_q.restype = Z
    lib.mla_decode_plan_q.argtypes = [P, I, I, I, I, I, I, P, Z, P]
    lib.mla_decode_plan_q.restype = I
    lib.mla_decode_q.argtypes = [ctypes.POINTER(_Pool), I, P, P, P, I, P, I, I, I, ctypes.c_float, I,
                                 P, P, P, P]
    lib.mla_decode_q.restype = I
    L = ctypes.c_int64
    lib.mla_extend_tables.argtypes = [P, P, I, I, I, P, P, I, P, I, P, P, I, P, P, P, I, P, P, P]
    lib.mla_extend_tables.restype = I
    lib.mla_rope_write.argtypes = [ctypes.c_char_p, I, P, P, I, P, I, ctypes.c_char_p, P, I, I, P,
                                   ctypes.c_float, P, L, P, L, I, P, P]
    lib.mla_rope_write.restype = I
    lib.mla_prefill.argtypes = [ctypes.c_char_p, I, P, P, P, P, I, P, I, I, L, I, P, P, ctypes.c_float, I,
                                P, Z, P, P, P]
    lib.mla_prefill.restype = I
    lib.mla_prefill_workspace_size.argtypes = [I, I, L, I, I]
    lib.mla_prefill_workspace_size.restype = Z
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != MLA_OK:
        raise MlaError("%s failed: %s (%d)" % (what, ERRORS.get(rc, "unknown"), rc))


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    # (the handle alone: building a Stream object costs as much as a launch)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


@dataclass
class KVPool:
    """A paged latent pool [num_layers, num_pages, page_size, 576] of bf16 or
    e4m3 codes (torch.uint8), with the fp8 per-pool scale."""
    data: torch.Tensor
    kv_scale: float = 1.0

    @property
    def dtype_code(self) -> int:
        return DTYPE_BF16 if self.data.dtype == torch.bfloat16 else DTYPE_FP8_E4M3

    def _c(self) -> _Pool:
        d = self.data
        shape = d.shape
        if len(shape) != 4 or shape[3] != LATENT_DIM:
            raise ValueError("pool must be [num_layers, num_pages, page_size, 576]")
        dtype = d.dtype
        if dtype is not torch.bfloat16 and dtype is not torch.uint8:
            raise ValueError("pool dtype must be bfloat16 or uint8 (e4m3 codes)")
        return _Pool(_dev(d, "pool"), shape[0], shape[1], shape[2],
                     DTYPE_BF16 if dtype is torch.bfloat16 else DTYPE_FP8_E4M3, self.kv_scale)

    def _packed(self, device: int) -> bytes:
        """The same structure as bytes (quicker made than a ctypes one)."""
        d = self.data
        if d.dim() != 4 or d.size(3) != LATENT_DIM:
            raise ValueError("pool must be [num_layers, num_pages, page_size, 576]")
        code = DTYPE_BF16 if d.dtype is torch.bfloat16 else DTYPE_FP8_E4M3
        if code == DTYPE_FP8_E4M3 and d.dtype is not torch.uint8:
            raise ValueError("pool dtype must be bfloat16 or uint8 (e4m3 codes)")
        return _pack_pool(_here(d, "pool", None, device), d.size(0), d.size(1), d.size(2), code, self.kv_scale)


def kv_write(pool: KVPool, layer: int, new_rows: torch.Tensor, slot_mapping: torch.Tensor,
             workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    lib = load_library()
    n = new_rows.shape[0]
    if new_rows.dim() != 2 or new_rows.shape[1] != LATENT_DIM or slot_mapping.shape != (n,):
        raise ValueError("new_rows [n, 576] and slot_mapping [n] expected")
    c = pool._c()
    rc = lib.mla_kv_write(ctypes.byref(c), layer, _dev(new_rows, "new_rows", torch.bfloat16),
                          _dev(slot_mapping, "slot_mapping", torch.int64), n,
                          None if workspace is None else _dev(workspace, "workspace"),
                          _stream(stream))
    _check(rc, "mla_kv_write")


def num_clusters() -> int:
    rc = load_library().mla_decode_num_clusters()
    if rc < 0:
        _check(rc, "mla_decode_num_clusters")
    return rc


def workspace_size(batch: int, num_heads: int) -> int:
    n = load_library().mla_decode_workspace_size(batch, num_heads)
    if n == 0:
        raise MlaError("mla_decode_workspace_size: unsupported arguments")
    return n


def alloc_workspace(batch: int, num_heads: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor (torch allocations are 256-byte aligned)."""
    return torch.zeros(workspace_size(batch, num_heads), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def plan(context_lens: torch.Tensor, num_heads: int, page_size: int, window: int,
         workspace: torch.Tensor, num_clusters: int = 0, stream=None) -> None:
    lib = load_library()
    rc = lib.mla_decode_plan(_dev(context_lens, "context_lens", torch.int32), context_lens.numel(),
                             num_heads, page_size, window, num_clusters,
                             _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                             _stream(stream))
    _check(rc, "mla_decode_plan")


def decode(pool: KVPool, layer: int, q: torch.Tensor, context_lens: torch.Tensor,
           softmax_scale: float, workspace: torch.Tensor, out: torch.Tensor,
           block_table: Optional[torch.Tensor] = None, page_indptr: Optional[torch.Tensor] = None,
           page_ids: Optional[torch.Tensor] = None, window: int = 0,
           lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    lib = load_library()
    if q.dim() != 3 or q.shape[2] != LATENT_DIM:
        raise ValueError("q must be [batch, heads, 576]")
    B, H, _ = q.shape
    if out.shape != (B, H, KV_LORA_RANK):
        raise ValueError("out must be [batch, heads, 512]")
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [batch, max_blocks]")
        indptr_p, ids_p, max_blocks = None, _dev(block_table, "block_table", torch.int32), \
            block_table.shape[1]
    else:
        if page_indptr is None or page_ids is None or page_indptr.shape != (B + 1,):
            raise ValueError("give block_table, or page_indptr [batch+1] and page_ids")
        indptr_p = _dev(page_indptr, "page_indptr", torch.int32)
        ids_p, max_blocks = _dev(page_ids, "page_ids", torch.int32), 0
    if context_lens.shape != (B,):
        raise ValueError("context_lens must be [batch]")
    c = pool._c()
    rc = lib.mla_decode(ctypes.byref(c), layer, _dev(q, "q", torch.bfloat16), indptr_p, ids_p,
                        max_blocks, _dev(context_lens, "context_lens", torch.int32), B, H,
                        float(softmax_scale), window, _dev(workspace, "workspace"),
                        _dev(out, "out", torch.bfloat16),
                        None if lse is None else _dev(lse, "lse", torch.float32), _stream(stream))
    _check(rc, "mla_decode")
    return out


def uv_project(attn_out: torch.Tensor, w_uv: torch.Tensor, y: torch.Tensor,
               workspace: Optional[torch.Tensor] = None, stream=None):
    lib = load_library()
    B, H, D = attn_out.shape
    if D != KV_LORA_RANK or w_uv.shape != (H, KV_LORA_RANK, V_HEAD_DIM) or \
            y.shape != (B, H, V_HEAD_DIM):
        raise ValueError("attn_out [B,H,512], w_uv [H,512,128], y [B,H,128] expected")
    rc = lib.mla_uv_project(_dev(attn_out, "attn_out", torch.bfloat16),
                            _dev(w_uv, "w_uv", torch.bfloat16), _dev(y, "y", torch.bfloat16), B, H,
                            None if workspace is None else _dev(workspace, "workspace"),
                            _stream(stream))
    _check(rc, "mla_uv_project")
    return y


def decode_noalloc(pool: KVPool, layer: int, q: torch.Tensor, context_lens: torch.Tensor,
                   softmax_scale: float, out: torch.Tensor, block_table: torch.Tensor,
                   window: int = 0, num_clusters: int = 0, lse: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """mla_decode_plan + mla_decode without a caller workspace: the library's
    fixed scratch array holds the schedule and partials (see the C header for
    the size limit and the one-stream rule)."""
    lib = load_library()
    B, H, _ = q.shape
    c = pool._c()
    rc = lib.mla_decode_noalloc(ctypes.byref(c), layer, _dev(q, "q", torch.bfloat16), None,
                                _dev(block_table, "block_table", torch.int32), block_table.shape[1],
                                _dev(context_lens, "context_lens", torch.int32), B, H,
                                float(softmax_scale), window, num_clusters,
                                _dev(out, "out", torch.bfloat16),
                                None if lse is None else _dev(lse, "lse", torch.float32),
                                None if status is None else _dev(status, "status", torch.int32),
                                _stream(stream))
    _check(rc, "mla_decode_noalloc")
    return out


def get_error(workspace: torch.Tensor, clear: bool = False, stream=None) -> int:
    code = ctypes.c_int(0)
    rc = load_library().mla_get_error(_dev(workspace, "workspace"), ctypes.byref(code),
                                      1 if clear else 0, _stream(stream))
    _check(rc, "mla_get_error")
    return code.value


def selftest_bounded_wait(status: torch.Tensor, arrive: bool, limit_us: int, stream=None) -> None:
    """One thread waits on a fresh mbarrier for at most limit_us; without the
    arrival the wait runs out and MLA_STATUS_TIMEOUT is OR-ed into status
    (a device int32 tensor)."""
    if status.dtype != torch.int32 or status.numel() < 1:
        raise MlaError("mla_selftest_bounded_wait: status must be a device int32 tensor")
    rc = load_library().mla_selftest_bounded_wait(1 if arrive else 0, int(limit_us),
                                                  _dev(status, "status"), _stream(stream))
    _check(rc, "mla_selftest_bounded_wait")


# ----------------------------------------------------------------- several query positions per request

def workspace_size_q(batch: int, q_len: int, num_heads: int) -> int:
    n = load_library().mla_decode_workspace_size_q(batch, q_len, num_heads)
    if n == 0:
        raise MlaError("mla_decode_workspace_size_q: unsupported arguments")
    return n


def alloc_workspace_q(batch: int, q_len: int, num_heads: int, device=None) -> torch.Tensor:
    return torch.zeros(workspace_size_q(batch, q_len, num_heads), dtype=torch.uint8,
                       device=device or torch.device("cuda"))


def plan_q(context_lens: torch.Tensor, q_len: int, num_heads: int, page_size: int, window: int,
           workspace: torch.Tensor, num_clusters: int = 0, stream=None) -> None:
    lib = load_library()
    rc = lib.mla_decode_plan_q(_dev(context_lens, "context_lens", torch.int32), context_lens.numel(), q_len,
                               num_heads, page_size, window, num_clusters, _dev(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "mla_decode_plan_q")


def decode_q(pool: KVPool, layer: int, q: torch.Tensor, context_lens: torch.Tensor,
             softmax_scale: float, workspace: torch.Tensor, out: torch.Tensor,
             block_table: Optional[torch.Tensor] = None, page_indptr: Optional[torch.Tensor] = None,
             page_ids: Optional[torch.Tensor] = None, window: int = 0,
             lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """q [batch, q_len, heads, 576] -> out [batch, q_len, heads, 512] (lse
    [batch, q_len, heads]); query position i of request b attends positions
    up to context_lens[b] + i."""
    lib = load_library()
    if q.dim() != 4 or q.shape[3] != LATENT_DIM:
        raise ValueError("q must be [batch, q_len, heads, 576]")
    B, QL, H, _ = q.shape
    if out.shape != (B, QL, H, KV_LORA_RANK):
        raise ValueError("out must be [batch, q_len, heads, 512]")
    if lse is not None and lse.shape != (B, QL, H):
        raise ValueError("lse must be [batch, q_len, heads]")
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError("block_table must be [batch, max_blocks]")
        indptr_p, ids_p, max_blocks = None, _dev(block_table, "block_table", torch.int32), \
            block_table.shape[1]
    else:
        if page_indptr is None or page_ids is None or page_indptr.shape != (B + 1,):
            raise ValueError("give block_table, or page_indptr [batch+1] and page_ids")
        indptr_p = _dev(page_indptr, "page_indptr", torch.int32)
        ids_p, max_blocks = _dev(page_ids, "page_ids", torch.int32), 0
    if context_lens.shape != (B,):
        raise ValueError("context_lens must be [batch]")
    c = pool._c()
    rc = lib.mla_decode_q(ctypes.byref(c), layer, _dev(q, "q", torch.bfloat16), indptr_p, ids_p, max_blocks,
                          _dev(context_lens, "context_lens", torch.int32), B, QL, H, float(softmax_scale),
                          window, _dev(workspace, "workspace"), _dev(out, "out", torch.bfloat16),
                          None if lse is None else _dev(lse, "lse", torch.float32), _stream(stream))
    _check(rc, "mla_decode_q")
    return out


# ----------------------------------------------------------------- prefill step

_I32, _I64, _BF16, _F32 = torch.int32, torch.int64, torch.bfloat16, torch.float32


def _here(t: torch.Tensor, name: str, dtype, device: int) -> int:
    """Pointer of a contiguous tensor of `dtype` (None: any) on the current device."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device or (t.dtype is not dtype and dtype is not None) \
            or not t.is_contiguous():
        _dev(t, name, dtype)  # says what is wrong with it
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, t.get_device(), device))
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], name: str, dtype, device: int):
    return None if t is None else _here(t, name, dtype, device)


def extend_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, block_table: torch.Tensor, page_size: int, num_pages: int,
                  slot_mapping: torch.Tensor, q_indptr: torch.Tensor, state: torch.Tensor,
                  positions: Optional[torch.Tensor] = None, page_indptr: Optional[torch.Tensor] = None,
                  page_ids: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """Give new_lens[b] new tokens of each request their places: pages off the
    top of the stack free_pages[:free_count] into block_table, slots and
    positions of the tokens (-1 behind the last), their row pointers q_indptr,
    and the tables as CSR lists. state becomes (free pages left, first request
    refused for want of pages); it may share free_count's memory."""
    dev = torch.cuda.current_device()
    if context_lens.dim() != 1 or new_lens.dim() != 1 or new_lens.numel() != context_lens.numel():
        raise ValueError("context_lens and new_lens must be [batch]")
    B = context_lens.numel()
    if block_table.dim() != 2 or block_table.size(0) != B:
        raise ValueError("block_table must be [batch, max_blocks]")
    n = slot_mapping.numel()
    if slot_mapping.dim() != 1 or (positions is not None and (positions.dim() != 1 or positions.numel() != n)):
        raise ValueError("slot_mapping and positions must be [max_tokens]")
    if q_indptr.dim() != 1 or q_indptr.numel() != B + 1:
        raise ValueError("q_indptr must be [batch + 1]")
    if (page_indptr is None) != (page_ids is None):
        raise ValueError("give page_indptr and page_ids together")
    pi_p = ids_p = None
    max_ids = 0
    if page_indptr is not None:
        if page_indptr.dim() != 1 or page_indptr.numel() != B + 1:
            raise ValueError("page_indptr must be [batch + 1]")
        pi_p, ids_p = _here(page_indptr, "page_indptr", _I32, dev), _here(page_ids, "page_ids", _I32, dev)
        max_ids = page_ids.numel()
    if free_count.numel() < 1 or state.numel() < 2:
        raise ValueError("free_count needs one element and state two")
    rc = (_lib or load_library()).mla_extend_tables(
        _here(context_lens, "context_lens", _I32, dev), _here(new_lens, "new_lens", _I32, dev), B, page_size, num_pages,
        _here(free_pages, "free_pages", _I32, dev), _here(free_count, "free_count", _I32, dev), free_pages.numel(),
        _here(block_table, "block_table", _I32, dev), block_table.size(1),
        _here(slot_mapping, "slot_mapping", _I64, dev), None if positions is None else
        _here(positions, "positions", _I32, dev), n, _here(q_indptr, "q_indptr", _I32, dev), pi_p, ids_p, max_ids,
        _here(state, "state", _I32, dev), None if workspace is None else _here(workspace, "workspace", None, dev),
        _stream(stream))
    if rc:
        _check(rc, "mla_extend_tables")


def _head_rows(t: torch.Tensor, name: str, n: int, device: int):
    """Pointer, pitch and heads of the [tokens, heads, 64] rope dims of queries, a
    view whose (token, head) rows lie at one pitch."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        raise ValueError("%s must be a CUDA tensor on the current device" % name)
    if t.dtype is not _BF16 or t.dim() != 3 or t.size(0) != n or t.size(2) != ROPE_DIM:
        raise ValueError("%s must be bfloat16 [tokens, heads, 64]" % name)
    h = t.size(1)
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and n > 1 and s0 != h * s1):
        raise ValueError("%s: the (token, head) rows must lie at one pitch" % name)
    return t.data_ptr(), s1 if h > 1 else s0 if n > 1 else ROPE_DIM, h


def rope_write(pool: Optional[KVPool], layer: int, rows: Optional[torch.Tensor], slot_mapping: Optional[torch.Tensor],
               positions: torch.Tensor, cos_sin: torch.Tensor, norm_weight: Optional[torch.Tensor] = None,
               norm_eps: float = 1e-6, q_rope: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
               pair_axis=None, interleaved: bool = True, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """Rotate the rope dims of new latent rows and of their queries, normalise
    c_kv (norm_weight given) and store the rows at their slots. positions is
    [tokens] or [axes, tokens]; pair_axis gives each of the 32 pairs its axis.
    q_rope and q_out are views [tokens, heads, 64] of the queries' rope dims;
    q_out None rotates in place. rows None (with pool and slot_mapping as may
    be) rotates queries only."""
    dev = torch.cuda.current_device()
    pd = positions.dim()
    if pd == 2:
        axes, n = positions.size(0), positions.size(1)
    elif pd == 1:
        axes, n = 1, positions.size(0)
    else:
        raise ValueError("positions must be [tokens] or [axes, tokens]")
    if cos_sin.dim() != 2 or cos_sin.size(1) != ROPE_DIM:
        raise ValueError("cos_sin must be [positions, 64]")
    c = rows_p = slots_p = weight_p = qp = op = axis_of = None
    q_pitch = o_pitch = heads = 0
    if slot_mapping is not None:
        if slot_mapping.dim() != 1 or slot_mapping.numel() != n:
            raise ValueError("slot_mapping must be [tokens]")
        slots_p = _here(slot_mapping, "slot_mapping", _I64, dev)
    if rows is not None:
        if pool is None or slots_p is None or rows.dim() != 2 or rows.size(0) != n or rows.size(1) != LATENT_DIM:
            raise ValueError("rows [tokens, 576] go with pool and slot_mapping")
        rows_p = _here(rows, "rows", _BF16, dev)
        c = pool._packed(dev)
    if norm_weight is not None:
        if norm_weight.numel() != KV_LORA_RANK:
            raise ValueError("norm_weight must be [512]")
        weight_p = _here(norm_weight, "norm_weight", _BF16, dev)
    if pair_axis is not None:
        axis_of = bytes(pair_axis)
        if len(axis_of) != ROPE_DIM // 2:
            raise ValueError("pair_axis must name an axis for each of the 32 pairs")
    if q_rope is not None:
        qp, q_pitch, heads = _head_rows(q_rope, "q_rope", n, dev)
        if q_out is None:
            op, o_pitch = qp, q_pitch
        else:
            op, o_pitch, h2 = _head_rows(q_out, "q_out", n, dev)
            if h2 != heads:
                raise ValueError("q_rope and q_out must be [tokens, heads, 64]")
        if heads == 0:
            qp = op = None
    elif q_out is not None:
        raise ValueError("q_out goes with q_rope")
    elif rows is None:
        raise ValueError("give rows, q_rope or both")
    if n == 0 or (qp is None and rows_p is None):
        return
    rc = (_lib or load_library()).mla_rope_write(
        c, layer, rows_p, slots_p, n, _here(positions, "positions", _I32, dev), axes, axis_of,
        _here(cos_sin, "cos_sin", _F32, dev), cos_sin.size(0), 1 if interleaved else 0, weight_p, norm_eps, qp, q_pitch,
        op, o_pitch, heads, None if workspace is None else _here(workspace, "workspace", None, dev), _stream(stream))
    if rc:
        if axis_of is not None and max(axis_of) >= axes:
            raise ValueError("pair_axis names an axis that positions lacks")
        _check(rc, "mla_rope_write")


def prefill_workspace_size(batch: int, q_rows: int, max_kv_tokens: int, num_heads: int, heads_per_pass: int = 0) -> int:
    n = load_library().mla_prefill_workspace_size(batch, q_rows, max_kv_tokens, num_heads, heads_per_pass)
    if n == 0:
        raise MlaError("mla_prefill_workspace_size: unsupported arguments")
    return n


def alloc_prefill_workspace(batch: int, q_rows: int, max_kv_tokens: int, num_heads: int, heads_per_pass: int = 0,
                            device=None) -> torch.Tensor:
    """A workspace for prefill() with its status word cleared. heads_per_pass
    bounds its size: the keys and values of so many heads are kept at once."""
    ws = torch.empty(prefill_workspace_size(batch, q_rows, max_kv_tokens, num_heads, heads_per_pass),
                     dtype=torch.uint8, device=device or torch.device("cuda"))
    ws[:256].zero_()
    return ws


def prefill(pool: KVPool, layer: int, q: torch.Tensor, q_indptr: torch.Tensor, context_lens: torch.Tensor,
            softmax_scale: float, w_uk: torch.Tensor, w_uv: torch.Tensor, workspace: torch.Tensor, out: torch.Tensor,
            max_kv_tokens: int, block_table: Optional[torch.Tensor] = None,
            page_indptr: Optional[torch.Tensor] = None, page_ids: Optional[torch.Tensor] = None, window: int = 0,
            lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """q [rows, heads, 192] of ragged chunks (request b: rows q_indptr[b] to
    q_indptr[b + 1], at positions from context_lens[b]) -> out [rows, heads,
    128], lse [rows, heads]: causal attention over the paged cache, the new
    tokens' latent rows written beforehand."""
    dev = torch.cuda.current_device()
    if q.dim() != 3 or q.size(2) != QK_HEAD_DIM:
        raise ValueError("q must be [rows, heads, 192]")
    T, H = q.size(0), q.size(1)
    if out.shape != (T, H, V_HEAD_DIM) or (lse is not None and lse.shape != (T, H)):
        raise ValueError("out must be [rows, heads, 128], lse [rows, heads]")
    if context_lens.dim() != 1:
        raise ValueError("context_lens must be [batch]")
    B = context_lens.numel()
    if q_indptr.dim() != 1 or q_indptr.numel() != B + 1:
        raise ValueError("q_indptr must be [batch + 1]")
    if w_uk.shape != (H, NOPE_DIM, KV_LORA_RANK) or w_uv.shape != (H, KV_LORA_RANK, V_HEAD_DIM):
        raise ValueError("w_uk [heads, 128, 512] and w_uv [heads, 512, 128] expected")
    if block_table is not None:
        if block_table.dim() != 2 or block_table.size(0) != B:
            raise ValueError("block_table must be [batch, max_blocks]")
        indptr_p, ids_p, max_blocks = None, _here(block_table, "block_table", _I32, dev), block_table.size(1)
    else:
        if page_indptr is None or page_ids is None or page_indptr.dim() != 1 or page_indptr.numel() != B + 1:
            raise ValueError("give block_table, or page_indptr [batch+1] and page_ids")
        indptr_p, ids_p, max_blocks = _here(page_indptr, "page_indptr", _I32, dev), \
            _here(page_ids, "page_ids", _I32, dev), 0
    rc = (_lib or load_library()).mla_prefill(
        pool._packed(dev), layer, _here(q, "q", _BF16, dev), _here(q_indptr, "q_indptr", _I32, dev), indptr_p,
        ids_p, max_blocks, _here(context_lens, "context_lens", _I32, dev), B, T, max_kv_tokens, H,
        _here(w_uk, "w_uk", _BF16, dev), _here(w_uv, "w_uv", _BF16, dev), softmax_scale, window,
        _here(workspace, "workspace", None, dev), workspace.numel() * workspace.element_size(),
        _here(out, "out", _BF16, dev), _opt(lse, "lse", _F32, dev), _stream(stream))
    if rc:
        _check(rc, "mla_prefill")
    return out
