"""Thin ctypes binding of libsanta.so: argument marshalling only.

Every function takes torch CUDA tensors, checks their dtypes/shapes/layout, fills the C
structure declared in include/santa.h and calls the entry point of the same name on the
current torch stream.  All computation happens in the library's kernels; if the library
cannot be loaded, the first call raises (there is no CPU fallback).

Shapes (as in the C header): q [B][Hq][d]; k_pool, v_pool [P][Hkv][T][d] (float32 or
bfloat16); reps [P][Hkv][d] float32; page_table [B][max_teams] int32; seq_lens [B] int32.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import operator
import os
from dataclasses import dataclass

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))

DEV_BAD_PAGE, DEV_BAD_SEQLEN, DEV_BAD_SEL, DEV_TIMEOUT = 1, 2, 4, 8
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


class SantaError(RuntimeError):
    pass


class _DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
        ("reps", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("dtype", ctypes.c_int), ("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("team_size", ctypes.c_int),
        ("max_teams", ctypes.c_int), ("num_draws", ctypes.c_int),
        ("num_pages", ctypes.c_int64), ("seed", ctypes.c_uint64),
        ("out", ctypes.c_void_p), ("draw_ids", ctypes.c_void_p), ("sel_ids", ctypes.c_void_p),
        ("sel_count", ctypes.c_void_p), ("pi", ctypes.c_void_p), ("team_probs", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("device_status", ctypes.c_void_p),
        ("sampler", ctypes.c_int32), ("mix_alpha", ctypes.c_float),
    ]


class _AppendChunkArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p), ("rope", ctypes.c_void_p),
        ("rope_positions", ctypes.c_int64), ("num_tokens", ctypes.c_int64),
        ("num_pages", ctypes.c_int64), ("dtype", ctypes.c_int), ("batch", ctypes.c_int),
        ("num_q_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("team_size", ctypes.c_int), ("max_teams", ctypes.c_int),
        ("rope_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("q_out", ctypes.c_void_p),
        ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p), ("reps", ctypes.c_void_p),
        ("seq_lens_next", ctypes.c_void_p), ("device_status", ctypes.c_void_p),
    ]


class _ChunkArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("cu_q", ctypes.c_void_p), ("num_tokens", ctypes.c_int64), ("num_pages", ctypes.c_int64),
        ("dtype", ctypes.c_int), ("batch", ctypes.c_int), ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("team_size", ctypes.c_int),
        ("max_teams", ctypes.c_int), ("out", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("device_status", ctypes.c_void_p),
    ]


class _AppendNormArgs(ctypes.Structure):
    _fields_ = [
        ("chunk", _AppendChunkArgs), ("cache_type", ctypes.c_int), ("eps", ctypes.c_float),
        ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class _Q8Args(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("type", ctypes.c_int), ("window", ctypes.c_int),
        ("softcap", ctypes.c_float),
    ]


class _Q8ReadArgs(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p), ("first", ctypes.c_void_p), ("dst_table", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64), ("dst_pages", ctypes.c_int64), ("type", ctypes.c_int),
        ("out_dtype", ctypes.c_int), ("batch", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("team_size", ctypes.c_int), ("max_teams", ctypes.c_int),
        ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p),
        ("device_status", ctypes.c_void_p),
    ]


# Samplers (santa_sampler): i.i.d. draws with Horvitz-Thompson weights (the method),
# systematic draws with Horvitz-Thompson weights, i.i.d. draws with Hansen-Hurwitz weights.
SAMPLERS = {"iid_ht": 0, "systematic": 1, "iid_hh": 2}


_lib = None


def lib():
    """Load libsanta.so (building it from source first if it is missing or stale)."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        A = ctypes.POINTER(_DecodeArgs)
        sigs = {
            "santa_abi_version": (i32, []),
            "santa_status_string": (ctypes.c_char_p, [i32]),
            "santa_build_reps": (i32, [vp, i32, i64, i32, i32, i32, vp, vp, vp, vp]),
            "santa_update_reps": (i32, [vp, i32, i64, i32, i32, i32, vp, i32, vp, vp, vp, vp]),
            "santa_decode_workspace_bytes": (sz, [i32] * 8),
            "santa_decode_workspace_min_bytes": (sz, [i32] * 7),
            "santa_dense_workspace_bytes": (sz, [i32] * 7),
            "santa_sample": (i32, [A, vp]),
            "santa_attend_vs": (i32, [A, i32, vp, vp]),
            "santa_attend_vs_workspace_bytes": (sz, [i32] * 5),
            "santa_append_kv": (i32, [vp, vp, i32, i32, i32, i32, i32, i32, i64, vp, vp, vp, vp,
                                      vp, vp, vp, vp]),
            "santa_attend": (i32, [A, vp]),
            "santa_decode": (i32, [A, vp]),
            "santa_dense_decode": (i32, [A, vp]),
            "santa_decode_noalloc": (i32, [A, vp]),
            "santa_decode_host": (i32, [A, vp, vp, sz, vp, vp, sz, vp]),
            "santa_host_copy_route": (i32, [vp, vp, sz]),
            "santa_decode_plan": (i32, [A, i32, vp]),
            "santa_decode_path": (i32, [A]),
            "santa_noalloc_scratch_bytes": (sz, []),
            "santa_rope_table": (i32, [vp, i64, i32, ctypes.c_double, vp]),
            "santa_append_chunk": (i32, [ctypes.POINTER(_AppendChunkArgs), vp]),
            "santa_chunk_workspace_bytes": (sz, [i32, i32, i64] + [i32] * 5),
            "santa_chunk_attend": (i32, [ctypes.POINTER(_ChunkArgs), vp]),
            "santa_select_topk": (i32, [A, vp]),
            "santa_topk_decode": (i32, [A, vp]),
            "santa_append_norm": (i32, [ctypes.POINTER(_AppendNormArgs), vp]),
            "santa_q8_workspace_bytes": (sz, [i32] * 6),
            "santa_q8_dense_decode": (i32, [A, ctypes.POINTER(_Q8Args), vp]),
            "santa_q8_attend": (i32, [A, ctypes.POINTER(_Q8Args), vp]),
            "santa_q8_topk_decode": (i32, [A, ctypes.POINTER(_Q8Args), vp]),
            "santa_q8_decode": (i32, [A, ctypes.POINTER(_Q8Args), vp]),
            "santa_q8_read": (i32, [ctypes.POINTER(_Q8ReadArgs), vp]),
        }
        for name, (res, args) in sigs.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def santa_abi_version() -> int:
    return lib().santa_abi_version()


def santa_status_string(status: int) -> str:
    return lib().santa_status_string(status).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise SantaError(f"{what}: {santa_status_string(rc)} (status {rc})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _req(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SantaError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise SantaError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise SantaError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise SantaError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


def _dtype_code(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    return _DTYPES[dtype]


def santa_decode_workspace_bytes(dtype, batch, num_q_heads, num_kv_heads, head_dim, team_size,
                                 max_teams, num_draws) -> int:
    """dtype: torch.float32 / torch.bfloat16 (or 0 / 1)."""
    return lib().santa_decode_workspace_bytes(_dtype_code(dtype), batch, num_q_heads,
                                              num_kv_heads, head_dim, team_size, max_teams,
                                              num_draws)


def santa_decode_workspace_min_bytes(batch, num_q_heads, num_kv_heads, head_dim, team_size,
                                     max_teams, num_draws) -> int:
    return lib().santa_decode_workspace_min_bytes(batch, num_q_heads, num_kv_heads, head_dim,
                                                  team_size, max_teams, num_draws)


def santa_dense_workspace_bytes(dtype, batch, num_q_heads, num_kv_heads, head_dim, team_size,
                                max_teams) -> int:
    return lib().santa_dense_workspace_bytes(_dtype_code(dtype), batch, num_q_heads,
                                             num_kv_heads, head_dim, team_size, max_teams)


def santa_build_reps(k_pool: torch.Tensor, page_fill: torch.Tensor | None = None,
                     reps: torch.Tensor | None = None, device_status: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Mean key of every (page, KV head) -> reps [P][Hkv][d] float32."""
    _req(k_pool, "k_pool", ndim=4)
    P, Hkv, T, d = k_pool.shape
    if k_pool.dtype not in _DTYPES:
        raise SantaError("k_pool must be float32 or bfloat16")
    if reps is None:
        reps = torch.empty((P, Hkv, d), dtype=torch.float32, device=k_pool.device)
    _req(reps, "reps", torch.float32)
    if page_fill is not None:
        _req(page_fill, "page_fill", torch.int32)
    _check(lib().santa_build_reps(_ptr(k_pool), _DTYPES[k_pool.dtype], P, Hkv, T, d,
                                  _ptr(page_fill), _ptr(reps), _ptr(device_status),
                                  _stream(stream)), "santa_build_reps")
    return reps


def santa_update_reps(k_pool: torch.Tensor, pages: torch.Tensor, reps: torch.Tensor,
                      page_fill: torch.Tensor | None = None,
                      device_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Recompute the representatives of the listed pages in place."""
    _req(k_pool, "k_pool", ndim=4)
    _req(pages, "pages", torch.int32, 1)
    _req(reps, "reps", torch.float32)
    P, Hkv, T, d = k_pool.shape
    _check(lib().santa_update_reps(_ptr(k_pool), _DTYPES[k_pool.dtype], P, Hkv, T, d,
                                   _ptr(pages), pages.numel(), _ptr(page_fill), _ptr(reps),
                                   _ptr(device_status), _stream(stream)), "santa_update_reps")
    return reps


def _carve(slab: torch.Tensor, specs):
    """Views of a flat uint8 tensor: one per (shape, dtype) in specs, each starting on a
    16-byte boundary, in order."""
    views, off = [], 0
    for shape, dtype in specs:
        n = 1
        for x in shape:
            n *= x
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        views.append(slab[off:off + nbytes].view(dtype).view(shape))
        off += (nbytes + 15) // 16 * 16
    return views


def _packed_bytes(specs) -> int:
    total = 0
    for shape, dtype in specs:
        n = 1
        for x in shape:
            n *= x
        total += (n * torch.empty((), dtype=dtype).element_size() + 15) // 16 * 16
    return total


def _host_slab(nbytes: int) -> torch.Tensor:
    """Page-locked when a GPU is present (asynchronous copies), plain memory otherwise."""
    return torch.empty(nbytes, dtype=torch.uint8, pin_memory=torch.cuda.is_available())


def _output_specs(batch, num_q_heads, num_kv_heads, head_dim, num_draws):
    """out, draw_ids, sel_ids, sel_count, pi and the device status word."""
    B, Hkv, M = batch, num_kv_heads, max(num_draws, 1)
    return [((B, num_q_heads, head_dim), torch.float32), ((B, Hkv, M), torch.int32),
            ((B, Hkv, M), torch.int32), ((B, Hkv), torch.int32), ((B, Hkv, M), torch.float32),
            ((1,), torch.int32)]


def _output_views(batch, num_q_heads, num_kv_heads, head_dim, num_draws, device, packed):
    """(out, draw_ids, sel_ids, sel_count, pi, device_status) and their slab (None unless
    packed).  The status word starts at zero."""
    specs = _output_specs(batch, num_q_heads, num_kv_heads, head_dim, num_draws)
    if not packed:
        views = [torch.empty(shape, dtype=dt, device=device) for shape, dt in specs[:-1]]
        return views + [torch.zeros(1, dtype=torch.int32, device=device)], None
    slab = torch.zeros(_packed_bytes(specs), dtype=torch.uint8, device=device)
    return _carve(slab, specs), slab


@dataclass
class HostOutputs:
    """Host copies of a packed DecodeBuffers' outputs and status word (views of `slab`)."""
    out: torch.Tensor
    draw_ids: torch.Tensor
    sel_ids: torch.Tensor
    sel_count: torch.Tensor
    pi: torch.Tensor
    device_status: torch.Tensor
    slab: torch.Tensor


@dataclass
class DecodeBuffers:
    """Outputs and scratch of one decode step for a fixed shape (reusable across steps)."""
    out: torch.Tensor          # [B][Hq][d] float32
    draw_ids: torch.Tensor     # [B][Hkv][M] int32
    sel_ids: torch.Tensor      # [B][Hkv][M] int32
    sel_count: torch.Tensor    # [B][Hkv] int32
    pi: torch.Tensor           # [B][Hkv][M] float32
    team_probs: torch.Tensor | None   # [B][Hkv][max_teams] float32
    workspace: torch.Tensor    # uint8
    device_status: torch.Tensor  # [1] int32
    outputs: torch.Tensor | None = None   # packed: the five outputs above as one uint8 slab

    @staticmethod
    def allocate(dtype, batch, num_q_heads, num_kv_heads, head_dim, team_size, max_teams,
                 num_draws, device="cuda", team_probs=False, dense=False,
                 packed=False) -> "DecodeBuffers":
        """dtype of q/K/V (torch.float32 or torch.bfloat16); sizes as in santa.h.  With
        packed=True, out, draw_ids, sel_ids, sel_count, pi and device_status are views of one
        slab (`outputs`, each view 16-byte aligned), so one copy brings them all to the host
        (host_mirror / download)."""
        B, Hkv, M = batch, num_kv_heads, max(num_draws, 1)
        ws = (santa_dense_workspace_bytes(dtype, B, num_q_heads, Hkv, head_dim, team_size,
                                          max_teams)
              if dense else
              santa_decode_workspace_bytes(dtype, B, num_q_heads, Hkv, head_dim, team_size,
                                           max_teams, M))
        if ws == 0:
            raise SantaError("unsupported shape for the workspace query")
        views, slab = _output_views(B, num_q_heads, Hkv, head_dim, M, device, packed)
        return DecodeBuffers(
            out=views[0], draw_ids=views[1], sel_ids=views[2], sel_count=views[3], pi=views[4],
            team_probs=(torch.empty((B, Hkv, max_teams), dtype=torch.float32, device=device)
                        if team_probs else None),
            workspace=torch.zeros(ws, dtype=torch.uint8, device=device),
            device_status=views[5],
            outputs=slab,
        )

    def host_mirror(self) -> HostOutputs:
        """Host buffers with the packed layout of this DecodeBuffers (packed=True only)."""
        if self.outputs is None:
            raise SantaError("host_mirror needs DecodeBuffers.allocate(..., packed=True)")
        B, Hq, d = self.out.shape
        _, Hkv, M = self.pi.shape
        specs = _output_specs(B, Hq, Hkv, d, M)
        slab = _host_slab(self.outputs.numel())
        return HostOutputs(*_carve(slab, specs), slab=slab)

    def download(self, host: HostOutputs, stream=None) -> HostOutputs:
        """One asynchronous device->host copy of the outputs and status into `host` on `stream`
        (the current stream by default); synchronise before reading it."""
        if self.outputs is None or host.slab.numel() != self.outputs.numel():
            raise SantaError("download needs a packed DecodeBuffers and its host_mirror()")
        if stream is None:
            host.slab.copy_(self.outputs, non_blocking=True)
        else:
            with torch.cuda.stream(stream):
                host.slab.copy_(self.outputs, non_blocking=True)
        return host

    def status(self) -> int:
        """Synchronise with the device and return the device status word."""
        return int(self.device_status.item())


@dataclass
class StepInputs:
    """The per-step inputs q [B][Hq][d], page_table [B][max_teams] and seq_lens [B] as views
    of one device slab, with host buffers of the same layout (host_q, host_page_table,
    host_seq_lens), so that one copy uploads a step's inputs."""
    q: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    host_q: torch.Tensor
    host_page_table: torch.Tensor
    host_seq_lens: torch.Tensor
    slab: torch.Tensor
    host_slab: torch.Tensor

    @staticmethod
    def allocate(dtype, batch, num_q_heads, head_dim, max_teams, device="cuda") -> "StepInputs":
        specs = [((batch, num_q_heads, head_dim), dtype), ((batch, max_teams), torch.int32),
                 ((batch,), torch.int32)]
        nbytes = _packed_bytes(specs)
        slab = torch.empty(nbytes, dtype=torch.uint8, device=device)
        host = _host_slab(nbytes)
        return StepInputs(*_carve(slab, specs), *_carve(host, specs), slab=slab,
                          host_slab=host)

    def upload(self, stream=None) -> "StepInputs":
        """One asynchronous host->device copy of the three host buffers on `stream`."""
        if stream is None:
            self.slab.copy_(self.host_slab, non_blocking=True)
        else:
            with torch.cuda.stream(stream):
                self.slab.copy_(self.host_slab, non_blocking=True)
        return self


class PreparedDecode:
    """santa_decode with its arguments checked and marshalled once, for steps that reuse
    the same tensors (a decode loop over persistent buffers).  run(seed) changes only the
    seed; the tensors' contents may change between runs, their storage may not."""

    def __init__(self, q, k_pool, v_pool, reps, page_table, seq_lens, num_draws: int,
                 bufs: DecodeBuffers | None = None, sampler: str = "iid_ht",
                 mix_alpha: float = 0.0, team_probs: bool = False):
        self.bufs = _bufs_for(q, k_pool, page_table, num_draws, bufs, team_probs)
        self._keep = (q, k_pool, v_pool, reps, page_table, seq_lens)
        self._a = _args(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws, 0,
                        self.bufs, sampler, mix_alpha)
        self._fn = lib().santa_decode
        self._aref = ctypes.byref(self._a)
        self._host_call = None      # (inputs, host, santa_decode_host's buffer arguments)

    def run(self, seed: int, stream=None) -> DecodeBuffers:
        self._a.seed = seed & 0xFFFFFFFFFFFFFFFF
        _check(self._fn(self._aref, _stream(stream)), "santa_decode")
        return self.bufs

    def run_host(self, seed: int, inputs: StepInputs, host: HostOutputs,
                 stream=None) -> HostOutputs:
        """One step through santa_decode_host: inputs.host_slab -> inputs.slab, the decode,
        bufs.outputs -> host.slab, then a wait for the stream.  The PreparedDecode must have
        been made on inputs' device views and packed DecodeBuffers; host.device_status holds
        the step's status word (sticky: zero it in the device slab to clear it)."""
        c = self._host_call
        if c is None or c[0] is not inputs or c[1] is not host:
            b = self.bufs
            if (b.outputs is None or host.slab.numel() != b.outputs.numel() or
                    self._a.q != inputs.q.data_ptr() or
                    self._a.page_table != inputs.page_table.data_ptr() or
                    self._a.seq_lens != inputs.seq_lens.data_ptr()):
                raise SantaError("run_host needs packed DecodeBuffers, their host_mirror() "
                                 "and a PreparedDecode made on the StepInputs' device views")
            # checked once per (inputs, host) pair: their storage may not change afterwards
            c = self._host_call = (inputs, host, lib().santa_decode_host,
                                   (inputs.host_slab.data_ptr(), inputs.slab.data_ptr(),
                                    inputs.slab.numel(), host.slab.data_ptr(),
                                    b.outputs.data_ptr(), b.outputs.numel()))
        self._a.seed = seed & 0xFFFFFFFFFFFFFFFF
        _check(c[2](self._aref, *c[3], _stream(stream)), "santa_decode_host")
        return host


def santa_decode_prepared(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws: int,
                          bufs: DecodeBuffers | None = None, sampler: str = "iid_ht",
                          mix_alpha: float = 0.0, team_probs: bool = False) -> PreparedDecode:
    """A PreparedDecode: santa_decode's checks and argument structure done once."""
    return PreparedDecode(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws, bufs,
                          sampler, mix_alpha, team_probs)


def _args(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws, seed,
          bufs: DecodeBuffers, sampler: str = "iid_ht", mix_alpha: float = 0.0) -> _DecodeArgs:
    _req(q, "q", ndim=3)
    _req(k_pool, "k_pool", ndim=4)
    _req(v_pool, "v_pool", ndim=4)
    _req(page_table, "page_table", torch.int32, 2)
    _req(seq_lens, "seq_lens", torch.int32, 1)
    if q.dtype not in _DTYPES or k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise SantaError("q, k_pool and v_pool must share one dtype (float32 or bfloat16)")
    if k_pool.shape != v_pool.shape:
        raise SantaError("k_pool and v_pool must have the same shape")
    if reps is not None:
        _req(reps, "reps", torch.float32, 3)
    B, Hq, d = q.shape
    P, Hkv, T, d2 = k_pool.shape
    if d2 != d or page_table.shape[0] != B or seq_lens.shape[0] != B:
        raise SantaError("shape mismatch between q, k_pool, page_table and seq_lens")
    a = _DecodeArgs()
    a.q, a.k_pool, a.v_pool, a.reps = _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(reps)
    a.page_table, a.seq_lens = _ptr(page_table), _ptr(seq_lens)
    a.dtype, a.batch, a.num_q_heads, a.num_kv_heads = _DTYPES[q.dtype], B, Hq, Hkv
    a.head_dim, a.team_size, a.max_teams, a.num_draws = d, T, page_table.shape[1], num_draws
    a.num_pages, a.seed = P, seed & 0xFFFFFFFFFFFFFFFF
    a.out, a.draw_ids, a.sel_ids = _ptr(bufs.out), _ptr(bufs.draw_ids), _ptr(bufs.sel_ids)
    a.sel_count, a.pi, a.team_probs = _ptr(bufs.sel_count), _ptr(bufs.pi), _ptr(bufs.team_probs)
    a.workspace, a.workspace_bytes = _ptr(bufs.workspace), bufs.workspace.numel()
    if sampler not in SAMPLERS:
        raise SantaError(f"unknown sampler {sampler!r} (one of {sorted(SAMPLERS)})")
    a.sampler, a.mix_alpha = SAMPLERS[sampler], float(mix_alpha)
    a.device_status = _ptr(bufs.device_status)
    return a


def _bufs_for(q, k_pool, page_table, num_draws, bufs, team_probs=False, dense=False):
    if bufs is not None:
        return bufs
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_pool.shape
    return DecodeBuffers.allocate(q.dtype, B, Hq, Hkv, d, T, page_table.shape[1], num_draws,
                                  q.device, team_probs=team_probs, dense=dense)


def santa_append_kv(k_new, v_new, k_pool, v_pool, reps, page_table, seq_lens,
                    seq_lens_next: torch.Tensor | None = None,
                    device_status: torch.Tensor | None = None, stream=None):
    """Write one new token per (sequence, KV head) (k_new, v_new [B][Hkv][d]) at position
    seq_lens[b] of the paged cache and refresh its page's representative; seq_lens_next (if
    given) receives seq_lens + 1.  All tensors on the device; nothing is allocated."""
    _req(k_new, "k_new", ndim=3)
    _req(v_new, "v_new", ndim=3)
    _req(k_pool, "k_pool", ndim=4)
    _req(reps, "reps", torch.float32, 3)
    _req(page_table, "page_table", torch.int32, 2)
    _req(seq_lens, "seq_lens", torch.int32, 1)
    if seq_lens_next is not None:
        _req(seq_lens_next, "seq_lens_next", torch.int32, 1)
    if k_new.dtype not in _DTYPES or {k_new.dtype, v_new.dtype, k_pool.dtype, v_pool.dtype} != {k_new.dtype}:
        raise SantaError("k_new, v_new, k_pool and v_pool must share one dtype")
    P, Hkv, T, d = k_pool.shape
    B = k_new.shape[0]
    if tuple(k_new.shape) != (B, Hkv, d) or tuple(v_new.shape) != (B, Hkv, d) or \
            tuple(v_pool.shape) != tuple(k_pool.shape):
        raise SantaError("k_new / v_new must be [B][Hkv][d] matching the pool")
    _check(lib().santa_append_kv(_ptr(k_new), _ptr(v_new), _DTYPES[k_new.dtype], B, Hkv, T, d,
                                 page_table.shape[1], P, _ptr(page_table), _ptr(seq_lens),
                                 _ptr(k_pool), _ptr(v_pool), _ptr(reps), _ptr(seq_lens_next),
                                 _ptr(device_status), _stream(stream)), "santa_append_kv")


def santa_sample(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws: int, seed: int,
                 bufs: DecodeBuffers | None = None, team_probs: bool = False,
                 stream=None, sampler: str = "iid_ht", mix_alpha: float = 0.0) -> DecodeBuffers:
    """Team distribution, M draws, distinct set and 1 / weight per selected team (the
    inclusion probability for the Horvitz-Thompson samplers)."""
    bufs = _bufs_for(q, k_pool, page_table, num_draws, bufs, team_probs)
    a = _args(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws, seed, bufs, sampler,
              mix_alpha)
    _check(lib().santa_sample(ctypes.byref(a), _stream(stream)), "santa_sample")
    return bufs


def santa_attend(q, k_pool, v_pool, page_table, seq_lens, sel_ids, sel_count, pi,
                 bufs: DecodeBuffers | None = None, stream=None) -> DecodeBuffers:
    """Horvitz-Thompson attention over the given teams (sel_ids [B][Hkv][M], sel_count
    [B][Hkv], pi [B][Hkv][M]); writes bufs.out."""
    _req(sel_ids, "sel_ids", torch.int32, 3)
    _req(sel_count, "sel_count", torch.int32, 2)
    _req(pi, "pi", torch.float32, 3)
    M = sel_ids.shape[2]
    bufs = _bufs_for(q, k_pool, page_table, M, bufs)
    a = _args(q, k_pool, v_pool, None, page_table, seq_lens, M, 0, bufs)
    a.sel_ids, a.sel_count, a.pi = _ptr(sel_ids), _ptr(sel_count), _ptr(pi)
    _check(lib().santa_attend(ctypes.byref(a), _stream(stream)), "santa_attend")
    return bufs


def santa_attend_vs(q, k_pool, v_pool, page_table, seq_lens, sel_ids, sel_count, pi,
                    value_rows: int, seed: int, bufs: DecodeBuffers | None = None,
                    value_ids: bool = False, stream=None):
    """Attention over the given teams with value-row sampling inside each (value_rows rows
    per team, drawn from the group-mean in-team softmax with key `seed`); writes bufs.out.
    Returns (bufs, value_ids [B][Hkv][M][value_rows] int32 or None)."""
    _req(sel_ids, "sel_ids", torch.int32, 3)
    _req(sel_count, "sel_count", torch.int32, 2)
    _req(pi, "pi", torch.float32, 3)
    B, Hq, d = q.shape
    Hkv = k_pool.shape[1]
    M = sel_ids.shape[2]
    bufs = _bufs_for(q, k_pool, page_table, M, bufs)
    need = lib().santa_attend_vs_workspace_bytes(B, Hq, Hkv, d, M)
    if need == 0:
        raise SantaError("unsupported shape for santa_attend_vs")
    ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    vids = (torch.empty((B, Hkv, M, value_rows), dtype=torch.int32, device=q.device)
            if value_ids else None)
    a = _args(q, k_pool, v_pool, None, page_table, seq_lens, M, seed, bufs)
    a.sel_ids, a.sel_count, a.pi = _ptr(sel_ids), _ptr(sel_count), _ptr(pi)
    a.workspace, a.workspace_bytes = _ptr(ws), need
    _check(lib().santa_attend_vs(ctypes.byref(a), value_rows, _ptr(vids), _stream(stream)),
           "santa_attend_vs")
    return bufs, vids


def santa_decode(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws: int, seed: int,
                 bufs: DecodeBuffers | None = None, team_probs: bool = False,
                 stream=None, sampler: str = "iid_ht", mix_alpha: float = 0.0) -> DecodeBuffers:
    """One SANTA++ decode step: sampling then weighted attention (Horvitz-Thompson by
    default; see SAMPLERS and the defensive mixture weight mix_alpha)."""
    bufs = _bufs_for(q, k_pool, page_table, num_draws, bufs, team_probs)
    a = _args(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws, seed, bufs, sampler,
              mix_alpha)
    _check(lib().santa_decode(ctypes.byref(a), _stream(stream)), "santa_decode")
    return bufs


def santa_decode_noalloc(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws: int,
                         seed: int, bufs: DecodeBuffers, stream=None) -> DecodeBuffers:
    """santa_decode with the library's built-in scratch instead of bufs.workspace, for
    callers that cannot allocate device memory at call time (the caller still provides the
    outputs in bufs, team_probs included if wanted; bufs.workspace is not used)."""
    a = _args(q, k_pool, v_pool, reps, page_table, seq_lens, num_draws, seed, bufs)
    _check(lib().santa_decode_noalloc(ctypes.byref(a), _stream(stream)), "santa_decode_noalloc")
    return bufs


_PLAN_MODES = {"decode": 0, "sample": 1, "attend": 2, "dense": 3}


def santa_decode_plan(q, k_pool, page_table, num_draws: int, which: str = "decode",
                      workspace_bytes: int | None = None) -> dict:
    """The launch shape the library picks: cluster size, clusters per unit, teams per CTA,
    the device's co-resident cluster count for that size, and whether the wide
    (one-CTA-per-SM) variant runs."""
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_pool.shape
    a = _DecodeArgs()
    a.dtype, a.batch, a.num_q_heads, a.num_kv_heads = _DTYPES[q.dtype], B, Hq, Hkv
    a.head_dim, a.team_size, a.max_teams, a.num_draws = d, T, page_table.shape[1], num_draws
    a.num_pages = k_pool.shape[0]
    if workspace_bytes is None:
        workspace_bytes = (santa_dense_workspace_bytes(q.dtype, B, Hq, Hkv, d, T,
                                                       page_table.shape[1])
                           if which == "dense" else
                           santa_decode_workspace_bytes(q.dtype, B, Hq, Hkv, d, T,
                                                        page_table.shape[1], num_draws))
    a.workspace = 256 if workspace_bytes else None        # only its size is read
    a.workspace_bytes = workspace_bytes
    out = (ctypes.c_int32 * 5)()
    _check(lib().santa_decode_plan(ctypes.byref(a), _PLAN_MODES[which], out), "santa_decode_plan")
    return {"cluster": out[0], "clusters_per_unit": out[1], "teams_per_cta": out[2],
            "max_active_clusters": out[3], "wide": bool(out[4])}


def santa_decode_path(q, k_pool, page_table, num_draws: int, sampler: str = "iid_ht",
                      mix_alpha: float = 0.0, workspace_bytes: int | None = None) -> str:
    """"compact" or "general": the form of the decode kernel santa_decode runs for these
    shapes and sampler settings (with the default workspace unless workspace_bytes)."""
    B, Hq, d = q.shape
    _, Hkv, T, _ = k_pool.shape
    a = _DecodeArgs()
    a.dtype, a.batch, a.num_q_heads, a.num_kv_heads = _DTYPES[q.dtype], B, Hq, Hkv
    a.head_dim, a.team_size, a.max_teams, a.num_draws = d, T, page_table.shape[1], num_draws
    a.num_pages = k_pool.shape[0]
    a.sampler, a.mix_alpha = SAMPLERS[sampler], float(mix_alpha)
    if workspace_bytes is None:
        workspace_bytes = santa_decode_workspace_bytes(q.dtype, B, Hq, Hkv, d, T,
                                                       page_table.shape[1], num_draws)
    a.workspace = 256 if workspace_bytes else None        # only its size is read
    a.workspace_bytes = workspace_bytes
    rc = lib().santa_decode_path(ctypes.byref(a))
    if rc < 0:
        _check(-rc, "santa_decode_path")
    return "compact" if rc == 1 else "general"


def santa_noalloc_scratch_bytes() -> int:
    return lib().santa_noalloc_scratch_bytes()


def santa_dense_decode(q, k_pool, v_pool, page_table, seq_lens,
                       bufs: DecodeBuffers | None = None, stream=None) -> DecodeBuffers:
    """Exact dense split-K decode attention over every token (the speed reference)."""
    bufs = _bufs_for(q, k_pool, page_table, 1, bufs, dense=True)
    a = _args(q, k_pool, v_pool, None, page_table, seq_lens, 1, 0, bufs)
    _check(lib().santa_dense_decode(ctypes.byref(a), _stream(stream)), "santa_dense_decode")
    return bufs


# ---------------------------------------------------------------- chunks and top-k

def _same_device(**tensors):
    """Every given tensor lives on the current CUDA device (the one a call runs on)."""
    cur = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is not None and t.device.index != cur:
            raise SantaError(f"{name} is on {t.device}, the current device is cuda:{cur}")


def _allocating(stream):
    """Context in which torch allocates for `stream` (None: the current stream), so that a
    buffer's memory is reused only after the stream's work on it."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _status_word(t):
    if t is not None:
        _req(t, "device_status", torch.int32)
        if t.numel() < 1:
            raise SantaError("device_status must hold one int32")


def _pools(k_pool, v_pool, dtype):
    _req(k_pool, "k_pool", dtype, 4)
    _req(v_pool, "v_pool", dtype, 4)
    if k_pool.shape != v_pool.shape:
        raise SantaError("k_pool and v_pool must have the same shape")
    return k_pool.shape


def _ragged(cu_q, page_table, seq_lens):
    """Checks the batch's int32 tensors; returns B."""
    _req(cu_q, "cu_q", torch.int32, 1)
    _req(page_table, "page_table", torch.int32, 2)
    _req(seq_lens, "seq_lens", torch.int32, 1)
    B = seq_lens.shape[0]
    if cu_q.shape[0] != B + 1 or page_table.shape[0] != B:
        raise SantaError("cu_q must be [B + 1], page_table [B][max_teams] and seq_lens [B]")
    return B


def _token_rows(t, name, dtype, heads, d):
    """[tokens][heads][d] whose rows are contiguous; returns the row stride in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SantaError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise SantaError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or t.shape[2] != d:
        raise SantaError(f"{name} must be [tokens][heads][{d}], got {tuple(t.shape)}")
    if t.shape[0] == 0:
        return t.shape[1] * d
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d):
        raise SantaError(f"the heads of one token of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * d


# The current stream's handle without a Stream object around it (several times faster).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Prepared:
    """A call whose arguments are checked and marshalled once, for steps that reuse the same
    tensors: their contents may change between runs, their storage may not.  The runs of one
    handle share its buffers (workspace and results): a run on another stream must wait for the
    run before it, and work at the same time takes a handle each.  A CUDA graph that captured a
    run uses the handle's buffers: keep the handle as long as the graph is replayed."""

    def __init__(self, name, args, keep, result, made=(), stream=None):
        self._name, self._fn = name, getattr(lib(), name)
        args = args if isinstance(args, tuple) else (args,)
        self._a, self._aref = args[0], tuple(ctypes.byref(a) for a in args)
        self._keep, self._result = keep, result
        self._device = torch.cuda.current_device()
        # tensors that the preparation made, and the streams that the allocator waits for before
        # it reuses their memory: the one they were made for, then those that _record names to it
        self._made = made
        self._known = {self._raw(stream)} if made else set()

    def _raw(self, stream):
        return _raw_stream(self._device) if stream is None else _stream(stream)

    def run(self, stream=None):
        """Enqueues the call on `stream` (the current stream by default); returns its result
        buffers.  Buffers that the preparation made are filled on the stream that was current
        then: another stream must wait for it before its first run.  The handle and those buffers
        may be dropped while runs are in flight (a stream given as a raw handle must outlive
        them); tensors that the caller gave are the caller's to keep until the runs are done."""
        if torch.cuda.current_device() != self._device:
            raise SantaError(f"{self._name} was prepared on cuda:{self._device}")
        raw = self._raw(stream)
        if self._made and raw not in self._known:
            self._record(raw, stream)
        rc = self._fn(*self._aref, raw)
        if rc:
            _check(rc, self._name)
        return self._result

    def _record(self, raw, stream):
        """Memory that the preparation made is reused only after the work that this stream has
        been given by the time it is freed."""
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream()
        for t in self._made:
            t.record_stream(stream)
        self._known.add(raw)


def santa_rope_table(positions: int, rope_dim: int, theta: float = 10000.0, device="cuda",
                     stream=None) -> torch.Tensor:
    """[positions][rope_dim] float32: cos(p theta^(-2j / rope_dim)), j < rope_dim / 2, then the
    sines; angles in 64 bits."""
    if torch.device(device).type != "cuda":
        raise SantaError("santa_rope_table makes a table on a CUDA device")
    if positions < 1 or rope_dim < 1:
        raise SantaError("positions and rope_dim must be positive")
    with _allocating(stream):
        table = torch.empty((positions, rope_dim), dtype=torch.float32, device=device)
    _same_device(table=table)
    _check(lib().santa_rope_table(_ptr(table), positions, rope_dim, float(theta),
                                  _stream(stream)), "santa_rope_table")
    return table


def _append_args(q, k_new, v_new, cu_q, pools, dt, reps, page_table, seq_lens, rope,
                 seq_lens_next, q_out, interleaved, device_status, stream, **more):
    """The argument structure of an append of dt tokens into `pools`, the tensors it points into,
    q_out and whether it was made here; `more`: further tensors of the call."""
    k_pool, v_pool = pools
    P, Hkv, T, d = k_pool.shape
    B = _ragged(cu_q, page_table, seq_lens)
    _req(reps, "reps", torch.float32, 3)
    if tuple(reps.shape) != (P, Hkv, d):
        raise SantaError("reps must be [P][Hkv][d] of the pools")
    a = _AppendChunkArgs()
    a.k_stride = _token_rows(k_new, "k_new", dt, Hkv, d)
    a.v_stride = _token_rows(v_new, "v_new", dt, Hkv, d)
    n, made = k_new.shape[0], ()
    if v_new.shape[0] != n:
        raise SantaError("k_new and v_new must hold the same tokens")
    if q is not None:
        a.q_stride = _token_rows(q, "q", dt, None, d)
        if q.shape[0] != n:
            raise SantaError("q and k_new must hold the same tokens")
        if q.shape[1] < 1:
            raise SantaError("q must have a head")
        if q_out is None:
            with _allocating(stream):
                # rows that belong to no sequence are not written
                q_out = torch.zeros((n, q.shape[1], d), dtype=dt, device=q.device)
            made = (q_out,)
        _req(q_out, "q_out", dt, 3)
        if q_out.shape != q.shape:
            raise SantaError("q_out must have q's shape")
        a.num_q_heads = q.shape[1]
    elif q_out is not None:
        raise SantaError("q_out without q")
    if rope is not None:
        _req(rope, "rope", torch.float32, 2)
        a.rope_positions, a.rope_dim = rope.shape
    if seq_lens_next is not None:
        _req(seq_lens_next, "seq_lens_next", torch.int32, 1)
        if seq_lens_next.shape[0] != B:
            raise SantaError("seq_lens_next must be [B]")
    _status_word(device_status)
    _same_device(q=q, k_new=k_new, v_new=v_new, cu_q=cu_q, k_pool=k_pool, v_pool=v_pool,
                 reps=reps, page_table=page_table, seq_lens=seq_lens, rope=rope, q_out=q_out,
                 seq_lens_next=seq_lens_next, device_status=device_status, **more)
    # an empty chunk has tensors without storage
    a.q, a.q_out = (_ptr(q), _ptr(q_out)) if n else (None, None)
    a.k_new, a.v_new = _ptr(k_new), _ptr(v_new)
    a.cu_q, a.page_table, a.seq_lens, a.rope = (_ptr(cu_q), _ptr(page_table), _ptr(seq_lens),
                                                _ptr(rope))
    a.num_tokens, a.num_pages, a.dtype, a.batch = n, P, _DTYPES[dt], B
    a.num_kv_heads, a.head_dim, a.team_size, a.max_teams = Hkv, d, T, page_table.shape[1]
    a.interleaved = int(bool(interleaved))
    a.k_pool, a.v_pool, a.reps = _ptr(k_pool), _ptr(v_pool), _ptr(reps)
    a.seq_lens_next, a.device_status = _ptr(seq_lens_next), _ptr(device_status)
    keep = (q, k_new, v_new, cu_q, k_pool, v_pool, reps, page_table, seq_lens, rope, q_out,
            seq_lens_next, device_status, *more.values())
    return a, keep, q_out, made


def _append_chunk(q, k_new, v_new, cu_q, k_pool, v_pool, reps, page_table, seq_lens, rope,
                  seq_lens_next, q_out, interleaved, device_status, stream):
    if not isinstance(k_pool, torch.Tensor) or k_pool.dtype not in _DTYPES:
        raise SantaError("k_pool must be a float32 or bfloat16 tensor")
    dt = k_pool.dtype
    _pools(k_pool, v_pool, dt)
    a, keep, q_out, made = _append_args(
        q, k_new, v_new, cu_q, (k_pool, v_pool), dt, reps, page_table, seq_lens, rope,
        seq_lens_next, q_out, interleaved, device_status, stream)
    return _Prepared("santa_append_chunk", a, keep, q_out, made, stream)


def santa_append_chunk(q, k_new, v_new, cu_q, k_pool, v_pool, reps, page_table, seq_lens,
                       rope: torch.Tensor | None = None,
                       seq_lens_next: torch.Tensor | None = None,
                       q_out: torch.Tensor | None = None, interleaved: bool = False,
                       device_status: torch.Tensor | None = None, stream=None):
    """A ragged chunk of new tokens (k_new, v_new [tokens][Hkv][d]; cu_q [B + 1]) into the paged
    cache behind seq_lens, keys and queries (q [tokens][Hq][d] or None) rotated by position with
    the table `rope` (None: not rotated), representatives of the touched pages refreshed;
    seq_lens_next (if given) receives the new lengths.  q, k_new and v_new may be strided from
    token to token (views of a fused projection).  Returns the rotated queries: q_out, or a new
    tensor whose rows outside every sequence are zero; q_out may be q itself if q is
    contiguous, and overlaps none of q, k_new and v_new otherwise."""
    return _append_chunk(q, k_new, v_new, cu_q, k_pool, v_pool, reps, page_table, seq_lens,
                         rope, seq_lens_next, q_out, interleaved, device_status,
                         stream).run(stream)


def santa_append_chunk_prepared(q, k_new, v_new, cu_q, k_pool, v_pool, reps, page_table,
                                seq_lens, rope: torch.Tensor | None = None,
                                seq_lens_next: torch.Tensor | None = None,
                                q_out: torch.Tensor | None = None, interleaved: bool = False,
                                device_status: torch.Tensor | None = None) -> _Prepared:
    """santa_append_chunk's checks and argument structure done once; .run(stream=None)."""
    return _append_chunk(q, k_new, v_new, cu_q, k_pool, v_pool, reps, page_table, seq_lens,
                         rope, seq_lens_next, q_out, interleaved, device_status, None)


def santa_chunk_workspace_bytes(dtype, batch, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                team_size, max_teams) -> int:
    """dtype: torch.float32 / torch.bfloat16 (or 0 / 1); 0 for an unsupported shape."""
    return lib().santa_chunk_workspace_bytes(_dtype_code(dtype), batch, num_tokens, num_q_heads,
                                             num_kv_heads, head_dim, team_size, max_teams)


def _chunk_attend(q, k_pool, v_pool, page_table, seq_lens, cu_q, out, workspace, device_status,
                  stream):
    _req(q, "q", ndim=3)
    if q.dtype not in _DTYPES:
        raise SantaError("q must be float32 or bfloat16")
    P, Hkv, T, d = _pools(k_pool, v_pool, q.dtype)
    B = _ragged(cu_q, page_table, seq_lens)
    n, Hq, d2 = q.shape
    if d2 != d:
        raise SantaError("q and the pools must have the same head size")
    if out is not None:
        _req(out, "out", q.dtype, 3)
        if out.shape != q.shape:
            raise SantaError("out must have q's shape")
    _status_word(device_status)
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, 1)
    _same_device(q=q, k_pool=k_pool, v_pool=v_pool, page_table=page_table, seq_lens=seq_lens,
                 cu_q=cu_q, out=out, workspace=workspace, device_status=device_status)
    made = []
    with _allocating(stream):
        if out is None:
            # rows that belong to no sequence are not written
            out = torch.zeros_like(q)
            made.append(out)
        if workspace is None:
            need = santa_chunk_workspace_bytes(q.dtype, B, n, Hq, Hkv, d, T,
                                               page_table.shape[1])
            if need == 0:
                raise SantaError("unsupported shape for santa_chunk_attend")
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            made.append(workspace)
    a = _ChunkArgs()
    a.q, a.k_pool, a.v_pool = _ptr(q), _ptr(k_pool), _ptr(v_pool)
    a.page_table, a.seq_lens, a.cu_q = _ptr(page_table), _ptr(seq_lens), _ptr(cu_q)
    a.num_tokens, a.num_pages, a.dtype, a.batch = n, P, _DTYPES[q.dtype], B
    a.num_q_heads, a.num_kv_heads, a.head_dim = Hq, Hkv, d
    a.team_size, a.max_teams = T, page_table.shape[1]
    a.out, a.workspace, a.workspace_bytes = _ptr(out), _ptr(workspace), workspace.numel()
    a.device_status = _ptr(device_status)
    keep = (q, k_pool, v_pool, page_table, seq_lens, cu_q, out, workspace, device_status)
    return _Prepared("santa_chunk_attend", a, keep, out, tuple(made), stream)


def santa_chunk_attend(q, k_pool, v_pool, page_table, seq_lens, cu_q,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       device_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Exact causal attention of a ragged chunk (q [tokens][Hq][d], cu_q [B + 1]; the last
    cu_q[b + 1] - cu_q[b] of sequence b's seq_lens[b] cached tokens) over the paged cache.
    Returns out [tokens][Hq][d] in q's dtype, which does not overlap q (a new tensor: zero outside
    every sequence)."""
    return _chunk_attend(q, k_pool, v_pool, page_table, seq_lens, cu_q, out, workspace,
                         device_status, stream).run(stream)


def santa_chunk_attend_prepared(q, k_pool, v_pool, page_table, seq_lens, cu_q,
                                out: torch.Tensor | None = None,
                                workspace: torch.Tensor | None = None,
                                device_status: torch.Tensor | None = None) -> _Prepared:
    """santa_chunk_attend's checks, buffers and argument structure done once;
    .run(stream=None)."""
    return _chunk_attend(q, k_pool, v_pool, page_table, seq_lens, cu_q, out, workspace,
                         device_status, None)


def _topk(name, q, k_pool, v_pool, reps, page_table, seq_lens, num_teams, bufs, stream):
    if reps is None:
        raise SantaError("reps must be a CUDA tensor")
    _req(k_pool, "k_pool", ndim=4)
    _req(q, "q", ndim=3)
    _req(page_table, "page_table", torch.int32, 2)
    if tuple(reps.shape) != (k_pool.shape[0], k_pool.shape[1], k_pool.shape[3]):
        raise SantaError("reps must be [P][Hkv][d] of the pools")
    made = ()
    if bufs is None:
        if q.dtype not in _DTYPES:
            raise SantaError("q must be float32 or bfloat16")
        _same_device(q=q)
        with _allocating(stream):
            bufs = _bufs_for(q, k_pool, page_table, num_teams, None)
        made = tuple(t for t in vars(bufs).values() if t is not None)
    B, Hq, d = q.shape
    Hkv = k_pool.shape[1]
    for field, shape, dt in (("out", (B, Hq, d), torch.float32),
                             ("sel_ids", (B, Hkv, num_teams), torch.int32),
                             ("sel_count", (B, Hkv), torch.int32),
                             ("pi", (B, Hkv, num_teams), torch.float32)):
        _req(getattr(bufs, field), f"bufs.{field}", dt)
        if tuple(getattr(bufs, field).shape) != shape:
            raise SantaError(f"bufs.{field} must be {shape}")
    a = _args(q, k_pool, v_pool, reps, page_table, seq_lens, num_teams, 0, bufs)
    _same_device(q=q, k_pool=k_pool, v_pool=v_pool, reps=reps, page_table=page_table,
                 seq_lens=seq_lens, out=bufs.out, sel_ids=bufs.sel_ids,
                 sel_count=bufs.sel_count, pi=bufs.pi, workspace=bufs.workspace,
                 device_status=bufs.device_status)
    # the buffers' tensors themselves: the fields of bufs may be replaced later
    keep = (q, k_pool, v_pool, reps, page_table, seq_lens, *vars(bufs).values())
    return _Prepared(name, a, keep, bufs, made, stream)


def santa_select_topk(q, k_pool, v_pool, reps, page_table, seq_lens, num_teams: int,
                      bufs: DecodeBuffers | None = None, stream=None) -> DecodeBuffers:
    """The num_teams teams of best representative score of every unit into bufs.sel_ids,
    bufs.sel_count and bufs.pi (1): the deterministic counterpart of santa_sample."""
    return _topk("santa_select_topk", q, k_pool, v_pool, reps, page_table, seq_lens, num_teams,
                 bufs, stream).run(stream)


def santa_topk_decode(q, k_pool, v_pool, reps, page_table, seq_lens, num_teams: int,
                      bufs: DecodeBuffers | None = None, stream=None) -> DecodeBuffers:
    """One sparse decode step: santa_select_topk, then exact attention inside those teams."""
    return _topk("santa_topk_decode", q, k_pool, v_pool, reps, page_table, seq_lens, num_teams,
                 bufs, stream).run(stream)


def santa_topk_decode_prepared(q, k_pool, v_pool, reps, page_table, seq_lens, num_teams: int,
                               bufs: DecodeBuffers | None = None) -> _Prepared:
    """santa_topk_decode's checks, buffers and argument structure done once;
    .run(stream=None)."""
    return _topk("santa_topk_decode", q, k_pool, v_pool, reps, page_table, seq_lens, num_teams,
                 bufs, None)


# ---------------------------------------------------------------- caches in 8 bits

_CODE_TYPES = {torch.int8: 2, torch.float8_e4m3fn: 3}


@dataclass
class Q8Cache:
    """A paged cache of 8-bit rows: codes k, v [P][Hkv][T][d] (int8 or float8_e4m3fn) and one
    scale for each row, k_scale, v_scale [P][Hkv][T] float32.  A row stands for codes * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @staticmethod
    def allocate(num_pages, num_kv_heads, team_size, head_dim, dtype=torch.int8,
                 device="cuda") -> "Q8Cache":
        """Rows of zeros."""
        if dtype not in _CODE_TYPES:
            raise SantaError("a cache of 8 bits is int8 or float8_e4m3fn")
        shape = (num_pages, num_kv_heads, team_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in "kv")
        k_scale, v_scale = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in "kv")
        return Q8Cache(k, v, k_scale, v_scale)

    def _check(self):
        """Checks the four tensors; returns [P][Hkv][T][d]."""
        if not isinstance(self.k, torch.Tensor) or self.k.dtype not in _CODE_TYPES:
            raise SantaError("cache.k must be an int8 or float8_e4m3fn tensor")
        _req(self.k, "cache.k", ndim=4)
        _req(self.v, "cache.v", self.k.dtype, 4)
        _req(self.k_scale, "cache.k_scale", torch.float32, 3)
        _req(self.v_scale, "cache.v_scale", torch.float32, 3)
        if self.v.shape != self.k.shape or self.k_scale.shape != self.k.shape[:3] or \
                self.v_scale.shape != self.k.shape[:3]:
            raise SantaError("a cache holds k and v [P][Hkv][T][d] and scales [P][Hkv][T]")
        return self.k.shape

    def _tensors(self):
        return dict(cache_k=self.k, cache_v=self.v, cache_k_scale=self.k_scale,
                    cache_v_scale=self.v_scale)


def _c_int(value, name) -> int:
    """A whole number that a C int holds (ctypes would keep its low 32 bits)."""
    try:
        x = operator.index(int(value) if isinstance(value, float) and value.is_integer() else value)
    except TypeError:
        raise SantaError(f"{name} must be a whole number, got {value!r}") from None
    if not -2**31 <= x < 2**31:
        raise SantaError(f"{name} = {x} does not fit 32 bits")
    return x


def _c_float(value, name) -> float:
    """A number that fp32 does not turn into zero or an infinity."""
    try:
        x = float(value)
    except (TypeError, ValueError, OverflowError):
        raise SantaError(f"{name} must be a number, got {value!r}") from None
    y = ctypes.c_float(x).value
    if (y == 0) != (x == 0) or math.isinf(y) != math.isinf(x):
        raise SantaError(f"{name} = {x} is out of fp32's range")
    return x


def _norm_weight(w, name, d):
    if w is not None:
        _req(w, name, torch.float32, 1)
        if w.shape[0] != d:
            raise SantaError(f"{name} must be [{d}]")


def _append_norm(q, k_new, v_new, cu_q, cache, reps, page_table, seq_lens, rope, q_norm, k_norm,
                 eps, seq_lens_next, q_out, interleaved, device_status, stream):
    a = _AppendNormArgs()
    if isinstance(cache, Q8Cache):
        cache._check()
        pools, scales = (cache.k, cache.v), (cache.k_scale, cache.v_scale)
        if not isinstance(k_new, torch.Tensor) or k_new.dtype not in _DTYPES:
            raise SantaError("k_new must be a float32 or bfloat16 tensor")
        dt = k_new.dtype
        a.cache_type = _CODE_TYPES[cache.k.dtype]
    else:
        if not isinstance(cache, (tuple, list)) or len(cache) != 2:
            raise SantaError("cache must be a Q8Cache or (k_pool, v_pool)")
        pools, scales = tuple(cache), (None, None)
        if not isinstance(pools[0], torch.Tensor) or pools[0].dtype not in _DTYPES:
            raise SantaError("k_pool must be a float32 or bfloat16 tensor")
        dt = pools[0].dtype
        _pools(*pools, dt)
        a.cache_type = _DTYPES[dt]
    a.eps = _c_float(eps, "eps")
    d = pools[0].shape[3]
    _norm_weight(q_norm, "q_norm", d)
    _norm_weight(k_norm, "k_norm", d)
    if q_norm is not None and q is None:
        raise SantaError("q_norm without q")
    a.chunk, keep, q_out, made = _append_args(
        q, k_new, v_new, cu_q, pools, dt, reps, page_table, seq_lens, rope, seq_lens_next, q_out,
        interleaved, device_status, stream, q_norm=q_norm, k_norm=k_norm, k_scale=scales[0],
        v_scale=scales[1])
    a.q_norm, a.k_norm = _ptr(q_norm), _ptr(k_norm)
    a.k_scale, a.v_scale = _ptr(scales[0]), _ptr(scales[1])
    return _Prepared("santa_append_norm", a, keep, q_out, made, stream)


def santa_append_norm(q, k_new, v_new, cu_q, cache, reps, page_table, seq_lens,
                      rope: torch.Tensor | None = None, q_norm: torch.Tensor | None = None,
                      k_norm: torch.Tensor | None = None, eps: float = 1e-6,
                      seq_lens_next: torch.Tensor | None = None,
                      q_out: torch.Tensor | None = None, interleaved: bool = False,
                      device_status: torch.Tensor | None = None, stream=None):
    """santa_append_chunk with the norms of the heads in the same pass (q_norm, k_norm: weights [d]
    float32 of x / sqrt(mean(x^2) + eps) * w for queries and keys, before the rotation; None: not
    normed), into `cache`: a Q8Cache, whose rows are rounded to 8 bits as they are written, or the
    pair (k_pool, v_pool) of the tokens' type."""
    return _append_norm(q, k_new, v_new, cu_q, cache, reps, page_table, seq_lens, rope, q_norm,
                        k_norm, eps, seq_lens_next, q_out, interleaved, device_status,
                        stream).run(stream)


def santa_append_norm_prepared(q, k_new, v_new, cu_q, cache, reps, page_table, seq_lens,
                               rope: torch.Tensor | None = None,
                               q_norm: torch.Tensor | None = None,
                               k_norm: torch.Tensor | None = None, eps: float = 1e-6,
                               seq_lens_next: torch.Tensor | None = None,
                               q_out: torch.Tensor | None = None, interleaved: bool = False,
                               device_status: torch.Tensor | None = None) -> _Prepared:
    """santa_append_norm's checks and argument structure done once; .run(stream=None)."""
    return _append_norm(q, k_new, v_new, cu_q, cache, reps, page_table, seq_lens, rope, q_norm,
                        k_norm, eps, seq_lens_next, q_out, interleaved, device_status, None)


def santa_q8_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, team_size,
                             max_teams) -> int:
    """Of the santa_q8_* attention; 0 for an unsupported shape."""
    return lib().santa_q8_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, team_size,
                                          max_teams)


def _q8_step(q, cache, page_table, seq_lens, softcap, window):
    """Checks and marshals what every attention over an 8-bit cache takes."""
    if not isinstance(cache, Q8Cache):
        raise SantaError("cache must be a Q8Cache")
    P, Hkv, T, d = cache._check()
    _req(q, "q", ndim=3)
    if q.dtype not in _DTYPES:
        raise SantaError("q must be float32 or bfloat16")
    _req(page_table, "page_table", torch.int32, 2)
    _req(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, d2 = q.shape
    if d2 != d or page_table.shape[0] != B or seq_lens.shape[0] != B:
        raise SantaError("shape mismatch between q, cache, page_table and seq_lens")
    a, c = _DecodeArgs(), _Q8Args()
    a.q, a.page_table, a.seq_lens = _ptr(q), _ptr(page_table), _ptr(seq_lens)
    a.dtype, a.batch, a.num_q_heads, a.num_kv_heads = _DTYPES[q.dtype], B, Hq, Hkv
    a.head_dim, a.team_size, a.max_teams, a.num_pages = d, T, page_table.shape[1], P
    c.k, c.v, c.k_scale, c.v_scale = (_ptr(cache.k), _ptr(cache.v), _ptr(cache.k_scale),
                                      _ptr(cache.v_scale))
    c.type, c.window, c.softcap = (_CODE_TYPES[cache.k.dtype], _c_int(window, "window"),
                                   _c_float(softcap, "softcap"))
    return a, c


def _q8_workspace(a, device):
    need = santa_q8_workspace_bytes(a.batch, a.num_q_heads, a.num_kv_heads, a.head_dim,
                                    a.team_size, a.max_teams)
    if need == 0:
        raise SantaError("unsupported shape for the attention over an 8-bit cache")
    return torch.empty(need, dtype=torch.uint8, device=device)


def _q8_attend(q, cache, page_table, seq_lens, sel, softcap, window, out, workspace,
               device_status, stream):
    a, c = _q8_step(q, cache, page_table, seq_lens, softcap, window)
    B, Hq, d = q.shape
    Hkv = cache.k.shape[1]
    name, lists = "santa_q8_dense_decode", {}
    if sel is not None:
        name = "santa_q8_attend"
        lists = dict(zip(("sel_ids", "sel_count", "pi"), sel))
        _req(lists["sel_ids"], "sel_ids", torch.int32, 3)
        _req(lists["sel_count"], "sel_count", torch.int32, 2)
        _req(lists["pi"], "pi", torch.float32, 3)
        M = lists["sel_ids"].shape[2]
        if tuple(lists["sel_ids"].shape) != (B, Hkv, M) or \
                tuple(lists["sel_count"].shape) != (B, Hkv) or \
                tuple(lists["pi"].shape) != (B, Hkv, M):
            raise SantaError("sel_ids and pi must be [B][Hkv][M] and sel_count [B][Hkv]")
        a.num_draws = M
        a.sel_ids, a.sel_count, a.pi = (_ptr(t) for t in lists.values())
    if out is not None:
        _req(out, "out", torch.float32, 3)
        if out.shape != q.shape:
            raise SantaError("out must have q's shape")
    if workspace is not None:
        _req(workspace, "workspace", torch.uint8, 1)
    _status_word(device_status)
    _same_device(q=q, page_table=page_table, seq_lens=seq_lens, out=out, workspace=workspace,
                 device_status=device_status, **cache._tensors(), **lists)
    made = []
    with _allocating(stream):
        if out is None:
            out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
            made.append(out)
        if workspace is None:
            workspace = _q8_workspace(a, q.device)
            made.append(workspace)
    a.out, a.workspace, a.workspace_bytes = _ptr(out), _ptr(workspace), workspace.numel()
    a.device_status = _ptr(device_status)
    keep = (q, page_table, seq_lens, out, workspace, device_status, *cache._tensors().values(),
            *lists.values())
    return _Prepared(name, (a, c), keep, out, tuple(made), stream)


def santa_q8_dense_decode(q, cache: Q8Cache, page_table, seq_lens, softcap: float = 0.0,
                          window: int = 0, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None,
                          device_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of one new token per sequence (q [B][Hq][d]) over every cached token of an 8-bit
    cache; softcap > 0: scores s become softcap * tanh(s / softcap); window > 0: the last `window`
    cached tokens only.  Returns out [B][Hq][d] float32."""
    return _q8_attend(q, cache, page_table, seq_lens, None, softcap, window, out, workspace,
                      device_status, stream).run(stream)


def santa_q8_dense_decode_prepared(q, cache: Q8Cache, page_table, seq_lens, softcap: float = 0.0,
                                   window: int = 0, out: torch.Tensor | None = None,
                                   workspace: torch.Tensor | None = None,
                                   device_status: torch.Tensor | None = None) -> _Prepared:
    """santa_q8_dense_decode's checks, buffers and argument structures done once;
    .run(stream=None)."""
    return _q8_attend(q, cache, page_table, seq_lens, None, softcap, window, out, workspace,
                      device_status, None)


def santa_q8_attend(q, cache: Q8Cache, page_table, seq_lens, sel_ids, sel_count, pi,
                    softcap: float = 0.0, window: int = 0, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None,
                    device_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """santa_attend over an 8-bit cache: the listed teams (sel_ids [B][Hkv][M], sel_count [B][Hkv])
    with weight 1 / pi [B][Hkv][M].  Returns out [B][Hq][d] float32."""
    return _q8_attend(q, cache, page_table, seq_lens, (sel_ids, sel_count, pi), softcap, window,
                      out, workspace, device_status, stream).run(stream)


def santa_q8_attend_prepared(q, cache: Q8Cache, page_table, seq_lens, sel_ids, sel_count, pi,
                             softcap: float = 0.0, window: int = 0,
                             out: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None,
                             device_status: torch.Tensor | None = None) -> _Prepared:
    """santa_q8_attend's checks, buffers and argument structures done once; .run(stream=None)."""
    return _q8_attend(q, cache, page_table, seq_lens, (sel_ids, sel_count, pi), softcap, window,
                      out, workspace, device_status, None)


def _q8_sparse(name, q, cache, reps, page_table, seq_lens, num_teams, softcap, window, bufs,
               stream, seed=0, sampler="iid_ht", mix_alpha=0.0):
    a, c = _q8_step(q, cache, page_table, seq_lens, softcap, window)
    if c.window:
        raise SantaError("the steps over best and sampled teams take no window (window must be 0)")
    P, Hkv, T, d = cache.k.shape
    B, Hq, _ = q.shape
    _req(reps, "reps", torch.float32, 3)
    if tuple(reps.shape) != (P, Hkv, d):
        raise SantaError("reps must be [P][Hkv][d] of the cache")
    if sampler not in SAMPLERS:
        raise SantaError(f"unknown sampler {sampler!r} (one of {sorted(SAMPLERS)})")
    made = ()
    if bufs is None:
        _same_device(q=q)
        with _allocating(stream):
            views, _ = _output_views(B, Hq, Hkv, d, num_teams, q.device, False)
            ws = _q8_workspace(a, q.device)
            # the arrival counters of the calls over 16- and 32-bit caches, which may get these buffers
            ws[:512 + 4 * B * Hkv].zero_()
            bufs = DecodeBuffers(*views[:5], None, ws, views[5])
        made = tuple(t for t in vars(bufs).values() if t is not None)
    fields = [("out", (B, Hq, d), torch.float32), ("sel_ids", (B, Hkv, num_teams), torch.int32),
              ("sel_count", (B, Hkv), torch.int32), ("pi", (B, Hkv, num_teams), torch.float32)]
    if name == "santa_q8_decode":
        fields.append(("draw_ids", (B, Hkv, num_teams), torch.int32))
        if bufs.team_probs is not None:
            fields.append(("team_probs", (B, Hkv, page_table.shape[1]), torch.float32))
    for field, shape, dt in fields:
        _req(getattr(bufs, field), f"bufs.{field}", dt)
        if tuple(getattr(bufs, field).shape) != shape:
            raise SantaError(f"bufs.{field} must be {shape}")
    _req(bufs.workspace, "bufs.workspace", torch.uint8, 1)
    _status_word(bufs.device_status)
    _same_device(q=q, reps=reps, page_table=page_table, seq_lens=seq_lens, **cache._tensors(),
                 **{f: getattr(bufs, f) for f, _, _ in fields}, workspace=bufs.workspace,
                 device_status=bufs.device_status)
    a.reps, a.num_draws, a.seed = _ptr(reps), num_teams, seed & 0xFFFFFFFFFFFFFFFF
    a.sampler, a.mix_alpha = SAMPLERS[sampler], float(mix_alpha)
    for field, _, _ in fields:
        setattr(a, field, _ptr(getattr(bufs, field)))
    a.workspace, a.workspace_bytes = _ptr(bufs.workspace), bufs.workspace.numel()
    a.device_status = _ptr(bufs.device_status)
    keep = (q, reps, page_table, seq_lens, *cache._tensors().values(), *vars(bufs).values())
    return _Prepared(name, (a, c), keep, bufs, made, stream)


def santa_q8_topk_decode(q, cache: Q8Cache, reps, page_table, seq_lens, num_teams: int,
                         softcap: float = 0.0, window: int = 0,
                         bufs: DecodeBuffers | None = None, stream=None) -> DecodeBuffers:
    """santa_topk_decode over an 8-bit cache: santa_select_topk, then santa_q8_attend.  window must
    be 0: teams are chosen from the whole sequence."""
    return _q8_sparse("santa_q8_topk_decode", q, cache, reps, page_table, seq_lens, num_teams,
                      softcap, window, bufs, stream).run(stream)


def santa_q8_topk_decode_prepared(q, cache: Q8Cache, reps, page_table, seq_lens, num_teams: int,
                                  softcap: float = 0.0, window: int = 0,
                                  bufs: DecodeBuffers | None = None) -> _Prepared:
    """santa_q8_topk_decode's checks, buffers and argument structures done once;
    .run(stream=None)."""
    return _q8_sparse("santa_q8_topk_decode", q, cache, reps, page_table, seq_lens, num_teams,
                      softcap, window, bufs, None)


def santa_q8_decode(q, cache: Q8Cache, reps, page_table, seq_lens, num_draws: int, seed: int,
                    softcap: float = 0.0, window: int = 0, bufs: DecodeBuffers | None = None,
                    stream=None, sampler: str = "iid_ht", mix_alpha: float = 0.0) -> DecodeBuffers:
    """santa_decode over an 8-bit cache: santa_sample, then santa_q8_attend.  window must be 0: teams
    are drawn from the whole sequence."""
    return _q8_sparse("santa_q8_decode", q, cache, reps, page_table, seq_lens, num_draws, softcap,
                      window, bufs, stream, seed, sampler, mix_alpha).run(stream)


def _q8_read(cache, page_table, seq_lens, k_out, v_out, dst_table, first, device_status, stream):
    if not isinstance(cache, Q8Cache):
        raise SantaError("cache must be a Q8Cache")
    P, Hkv, T, d = cache._check()
    if not isinstance(k_out, torch.Tensor) or k_out.dtype not in _DTYPES:
        raise SantaError("k_out must be a float32 or bfloat16 tensor")
    _req(k_out, "k_out", ndim=4)
    _req(v_out, "v_out", k_out.dtype, 4)
    if tuple(k_out.shape[1:]) != (Hkv, T, d) or v_out.shape != k_out.shape:
        raise SantaError("k_out and v_out must be [pages][Hkv][T][d] of the cache")
    _req(page_table, "page_table", torch.int32, 2)
    _req(dst_table, "dst_table", torch.int32, 2)
    _req(seq_lens, "seq_lens", torch.int32, 1)
    B = seq_lens.shape[0]
    if page_table.shape[0] != B or dst_table.shape != page_table.shape:
        raise SantaError("page_table and dst_table must be [B][max_teams] and seq_lens [B]")
    if first is not None:
        _req(first, "first", torch.int32, 1)
        if first.shape[0] != B:
            raise SantaError("first must be [B]")
    _status_word(device_status)
    _same_device(page_table=page_table, dst_table=dst_table, seq_lens=seq_lens, first=first,
                 k_out=k_out, v_out=v_out, device_status=device_status, **cache._tensors())
    a = _Q8ReadArgs()
    a.k, a.v, a.k_scale, a.v_scale = (_ptr(cache.k), _ptr(cache.v), _ptr(cache.k_scale),
                                      _ptr(cache.v_scale))
    a.page_table, a.seq_lens, a.first, a.dst_table = (_ptr(page_table), _ptr(seq_lens),
                                                      _ptr(first), _ptr(dst_table))
    a.num_pages, a.dst_pages, a.type, a.out_dtype = (P, k_out.shape[0], _CODE_TYPES[cache.k.dtype],
                                                     _DTYPES[k_out.dtype])
    a.batch, a.num_kv_heads, a.head_dim, a.team_size, a.max_teams = B, Hkv, d, T, page_table.shape[1]
    a.k_out, a.v_out, a.device_status = _ptr(k_out), _ptr(v_out), _ptr(device_status)
    keep = (page_table, dst_table, seq_lens, first, k_out, v_out, device_status,
            *cache._tensors().values())
    return _Prepared("santa_q8_read", a, keep, (k_out, v_out), (), stream)


def santa_q8_read(cache: Q8Cache, page_table, seq_lens, k_out, v_out, dst_table,
                  first: torch.Tensor | None = None, device_status: torch.Tensor | None = None,
                  stream=None):
    """Tokens first[b] (None: 0) .. seq_lens[b] - 1 of every sequence out of an 8-bit cache into the
    same slots of the pages that dst_table [B][max_teams] names in k_out, v_out [pages][Hkv][T][d]
    (float32 or bfloat16): a cache for santa_chunk_attend and the other calls.  Other slots are left
    as they were.  Returns (k_out, v_out)."""
    return _q8_read(cache, page_table, seq_lens, k_out, v_out, dst_table, first, device_status,
                    stream).run(stream)


def santa_q8_read_prepared(cache: Q8Cache, page_table, seq_lens, k_out, v_out, dst_table,
                           first: torch.Tensor | None = None,
                           device_status: torch.Tensor | None = None) -> _Prepared:
    """santa_q8_read's checks and argument structure done once; .run(stream=None)."""
    return _q8_read(cache, page_table, seq_lens, k_out, v_out, dst_table, first, device_status,
                    None)
