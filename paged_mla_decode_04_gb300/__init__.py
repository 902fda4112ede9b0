"""Paged MLA decode for GB300: thin Python binding of libmla_decode.so.

Argument marshalling only: every step runs in the library's CUDA kernels. (The
prefill step's calls, the shared prefixes' and the store's go through a compiled binding,
the others through ctypes.)
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
  plan_shared / decode_shared: decode of requests that share prefixes, each
  prefix attended once for its group
  quant_write / quant_read: a compact store of latent rows (QuantPool: e4m3 or
  4-bit codes with scales of their groups) and its way back
  get_error(workspace, clear=False)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from dataclasses import dataclass
from typing import Optional

import torch

from ._build import binding_path

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")
BINDING_PATH = binding_path()

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
            "mla_prefill", "mla_prefill_workspace_size", "mla_decode_workspace_size_shared",
            "mla_decode_plan_shared", "mla_decode_shared", "mla_quant_write", "mla_quant_read"]
NOALLOC_SCRATCH_BYTES = 48 << 20


class MlaError(RuntimeError):
    pass


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_layers", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("dtype", ctypes.c_int), ("kv_scale", ctypes.c_float)]


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
    lib.mla_decode_workspace_size_shared.argtypes = [I, I, I, I]
    lib.mla_decode_workspace_size_shared.restype = Z
    lib.mla_decode_plan_shared.argtypes = [P, P, P, I, I, I, I, I, I, P, Z, P]
    lib.mla_decode_plan_shared.restype = I
    lib.mla_decode_shared.argtypes = [ctypes.c_char_p, I, P, P, P, I, I, I, I, I, ctypes.c_float, P, P, P, P]
    lib.mla_decode_shared.restype = I
    lib.mla_quant_write.argtypes = [ctypes.c_char_p, I, P, P, I, P, P]
    lib.mla_quant_write.restype = I
    lib.mla_quant_read.argtypes = [ctypes.c_char_p, I, P, I, ctypes.c_char_p, I, P, P, P, P]
    lib.mla_quant_read.restype = I
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

_binding = None


def _step():
    """The compiled binding of these calls (see csrc/step_binding.cpp)."""
    global _binding
    if _binding is None:
        lib = load_library()
        if not os.path.exists(BINDING_PATH):
            raise MlaError("%s not built; run paged_mla_decode_04_gb300._build.build()" % os.path.basename(BINDING_PATH))
        spec = importlib.util.spec_from_file_location("_step_binding", BINDING_PATH)
        b = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(b)
        b.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (lib.mla_extend_tables, lib.mla_rope_write, lib.mla_prefill)])
        b.bind_shared(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.mla_decode_plan_shared, lib.mla_decode_shared, lib.mla_decode_workspace_size_shared, lib.mla_quant_write,
            lib.mla_quant_read)])
        _binding = b
    return _binding


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
    rc = (_binding or _step()).extend_tables(
        context_lens, new_lens, free_pages, free_count, block_table, page_size, num_pages, slot_mapping, q_indptr, state,
        positions, page_indptr, page_ids, workspace, stream)
    if rc:
        _check(rc, "mla_extend_tables")


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
    data, scale = (None, 1.0) if pool is None else (pool.data, pool.kv_scale)
    rc = (_binding or _step()).rope_write(
        data, scale, layer, rows, slot_mapping, positions, cos_sin, norm_weight, norm_eps, q_rope, q_out,
        None if pair_axis is None else bytes(pair_axis), interleaved, workspace, stream)
    if rc:
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
    rc = (_binding or _step()).prefill(
        pool.data, pool.kv_scale, layer, q, q_indptr, context_lens, softmax_scale, w_uk, w_uv, workspace, out,
        max_kv_tokens, block_table, page_indptr, page_ids, window, lse, stream)
    if rc:
        _check(rc, "mla_prefill")
    return out


# ----------------------------------------------------------------- shared prefixes

def workspace_size_shared(batch: int, q_len: int, num_heads: int, num_prefixes: int) -> int:
    n = load_library().mla_decode_workspace_size_shared(batch, q_len, num_heads, num_prefixes)
    if n == 0:
        raise MlaError("mla_decode_workspace_size_shared: unsupported arguments")
    return n


def alloc_workspace_shared(batch: int, q_len: int, num_heads: int, num_prefixes: int, device=None) -> torch.Tensor:
    """A workspace for plan_shared() and decode_shared() with its status word cleared."""
    ws = torch.empty(workspace_size_shared(batch, q_len, num_heads, num_prefixes), dtype=torch.uint8,
                     device=device or torch.device("cuda"))
    ws[:256].zero_()
    return ws


def plan_shared(context_lens: torch.Tensor, prefix_indptr: torch.Tensor, prefix_lens: torch.Tensor, q_len: int,
                num_heads: int, page_size: int, workspace: torch.Tensor, num_clusters: int = 0, stream=None) -> None:
    """The schedule of decode_shared() calls: requests prefix_indptr[g] to
    prefix_indptr[g + 1] share their first prefix_lens[g] cached positions."""
    rc = (_binding or _step()).plan_shared(context_lens, prefix_indptr, prefix_lens, q_len, num_heads, page_size, workspace,
                                           num_clusters, stream)
    if rc:
        _check(rc, "mla_decode_plan_shared")


def decode_shared(pool: KVPool, layer: int, q: torch.Tensor, num_prefixes: int, softmax_scale: float,
                  workspace: torch.Tensor, out: torch.Tensor, block_table: Optional[torch.Tensor] = None,
                  page_indptr: Optional[torch.Tensor] = None, page_ids: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """q [batch, q_len, heads, 576] -> out [batch, q_len, heads, 512] (lse [batch,
    q_len, heads]) as decode_q() without a window, each group's prefix read and
    attended once, by the plan in workspace."""
    rc = (_binding or _step()).decode_shared(
        pool.data, pool.kv_scale, layer, q, num_prefixes, softmax_scale, workspace, out, block_table, page_indptr, page_ids,
        lse, stream)
    if rc:
        _check(rc, "mla_decode_shared")
    return out


# ----------------------------------------------------------------- compact store

QUANT_E4M3_ROW = 656
QUANT_E2M1_ROW = 416


@dataclass
class QuantPool:
    """A compact store of latent rows [num_layers, num_pages, page_size, row bytes]
    of torch.uint8: 656 bytes a row (e4m3 codes, an fp32 scale for each 128 dims)
    or 416 (e2m1 codes, a bf16 scale for each 32 dims); the rope dims stay bf16."""
    data: torch.Tensor


def alloc_quant_pool(num_layers: int, num_pages: int, page_size: int, codes: str = "e4m3", device=None) -> QuantPool:
    """A store of zeros; codes "e4m3" or "e2m1"."""
    rows = {"e4m3": QUANT_E4M3_ROW, "e2m1": QUANT_E2M1_ROW}
    if codes not in rows:
        raise ValueError('codes must be "e4m3" or "e2m1"')
    return QuantPool(torch.zeros(num_layers, num_pages, page_size, rows[codes], dtype=torch.uint8,
                                 device=device or torch.device("cuda")))


def quant_write(store: QuantPool, layer: int, rows: torch.Tensor, slot_mapping: torch.Tensor,
                workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise latent rows [n, 576] into their slots [n] of the store."""
    rc = (_binding or _step()).quant_write(store.data, layer, rows, slot_mapping, workspace, stream)
    if rc:
        _check(rc, "mla_quant_write")


def quant_read(store: QuantPool, layer: int, slots: torch.Tensor, rows: Optional[torch.Tensor] = None,
               pool: Optional[KVPool] = None, pool_layer: int = 0, pool_slots: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Read slots [n] of the store back: into rows [n, 576], or into pool_slots [n] of
    a layer of a decode pool."""
    data, scale = (None, 1.0) if pool is None else (pool.data, pool.kv_scale)
    rc = (_binding or _step()).quant_read(store.data, layer, slots, rows, data, scale, pool_layer, pool_slots, workspace,
                                          stream)
    if rc:
        _check(rc, "mla_quant_read")
