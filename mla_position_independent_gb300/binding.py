"""Thin ctypes binding over libirm.so (include/irm.h).

Argument marshalling only: every step of the path runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  If libirm.so is missing the first
call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import torch

from .synth import CHUNK_DTYPE

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libirm.so")
_lib = None

WORKSPACE_HEADER = 256
DEFAULT_SCALE = 1.0 / math.sqrt(192.0)

EXPORTS = ["irm_status_string", "irm_last_error", "irm_version", "irm_validate_chunks",
           "irm_device_status", "irm_assemble_kv_workspace_size", "irm_assemble_kv",
           "irm_assemble_kv_rope", "irm_mla_attn_decode_workspace_size", "irm_mla_attn_decode",
           "irm_mla_attn_decode_rope", "irm_mla_attn_decode_noalloc", "irm_decode_noalloc_status",
           "irm_mla_attn_prefill_workspace_size", "irm_mla_attn_prefill", "irm_mla_attn_prefill_rope",
           "irm_cdc_sizes", "irm_cdc_chunk", "irm_registry_create", "irm_registry_stats",
           "irm_registry_assemble", "irm_selftest_wait_timeout", "irm_mla_attn_tree_workspace_size",
           "irm_mla_attn_tree", "irm_tree_verify", "irm_pages_workspace_size", "irm_pages_resize",
           "irm_pages_fork", "irm_pages_compact", "irm_pages_copy"]

ROPE_NEOX, ROPE_INTERLEAVED = 0, 1


class Rope(ctypes.Structure):
    """irm_rope: the model's RoPE variant (32 frequencies theta_j in radians per position and
    the pairing, ROPE_NEOX = dims (j, j+32) or ROPE_INTERLEAVED = dims (2j, 2j+1))."""
    _fields_ = [("inv_freq", ctypes.c_double * 32), ("pairing", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]

    @classmethod
    def make(cls, inv_freq, pairing=ROPE_NEOX):
        f = np.asarray(inv_freq, np.float64).reshape(32)
        return cls((ctypes.c_double * 32)(*f.tolist()), int(pairing), 0)


CDC_THRESHOLD, CDC_LOW_BITS = 0, 1


class CdcParams(ctypes.Structure):
    """irm_cdc_params: chunk length clip, boundary test and fingerprint seed."""
    _fields_ = [("min_len", ctypes.c_int32), ("max_len", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("seed", ctypes.c_uint64), ("gear_seed", ctypes.c_uint64)]

    @classmethod
    def make(cls, min_len=32, max_len=512, bits=7, mode=CDC_THRESHOLD, seed=0, gear_seed=0):
        return cls(int(min_len), int(max_len), int(bits), int(mode), int(seed), int(gear_seed))


def _rope_ptr(rope):
    return None if rope is None else ctypes.cast(ctypes.pointer(rope), ctypes.c_void_p)


class IrmError(RuntimeError):
    def __init__(self, status: int, text: str, detail: str):
        super().__init__(f"irm status {status} ({text}): {detail}")
        self.status = status


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built: run __graft_entry__.build() "
                               "(the CUDA library is required; there is no fallback)")
        L = ctypes.CDLL(_LIB_PATH)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.irm_status_string.restype = ctypes.c_char_p
        L.irm_status_string.argtypes = [I]
        L.irm_last_error.restype = ctypes.c_char_p
        L.irm_version.restype = ctypes.c_char_p
        L.irm_validate_chunks.argtypes = [P, P, I, I64, P]
        L.irm_device_status.argtypes = [P, P]
        L.irm_selftest_wait_timeout.argtypes = [P, SZ, P]
        L.irm_assemble_kv_workspace_size.argtypes = [P, P, I, P]
        L.irm_assemble_kv.argtypes = [P, P, I, P, I64, P, I64, P, I, P, P, P, P, SZ, P]
        L.irm_mla_attn_decode_workspace_size.argtypes = [P, P, I, I, P]
        L.irm_mla_attn_decode.argtypes = [P, P, I, I, P, P, P, I64, ctypes.c_float, P, P, P, SZ, P]
        L.irm_mla_attn_decode_noalloc.argtypes = [P, P, I, I, P, P, P, I64, ctypes.c_float, P, P, P]
        L.irm_decode_noalloc_status.argtypes = [P]
        L.irm_mla_attn_prefill_workspace_size.argtypes = [P, P, I, I, I, P]
        L.irm_mla_attn_prefill.argtypes = [P, P, I, I, I, P, P, P, I64, ctypes.c_float, P, P, P,
                                           SZ, P]
        L.irm_assemble_kv_rope.argtypes = [P, P, I, P, I64, P, I64, P, I, P, P, P, P, P, SZ, P]
        L.irm_mla_attn_decode_rope.argtypes = [P, P, I, I, P, P, P, I64, ctypes.c_float, P, P, P,
                                               P, SZ, P]
        L.irm_mla_attn_prefill_rope.argtypes = [P, P, I, I, I, P, P, P, I64, ctypes.c_float, P, P,
                                                P, P, SZ, P]
        L.irm_cdc_sizes.argtypes = [P, I, P, P, P]
        L.irm_cdc_chunk.argtypes = [P, P, I, P, ctypes.c_int32, P, P, P, P, P, P, SZ, P]
        L.irm_registry_create.argtypes = [I64, I64, I64, P]
        L.irm_registry_destroy.argtypes = [P]
        L.irm_registry_destroy.restype = None
        L.irm_registry_stats.argtypes = [P, P, P]
        L.irm_registry_assemble.argtypes = [P, P, I64, I64, I64, P, P, P, ctypes.c_int32, ctypes.c_int32,
                                            ctypes.c_uint64, P, P, ctypes.c_int32, P]
        L.irm_mla_attn_tree_workspace_size.argtypes = [P, P, I, I, P]
        L.irm_mla_attn_tree.argtypes = [P, P, I, I, P, P, P, I64, P, I, P, I, ctypes.c_float, P, P, P, SZ, P]
        L.irm_tree_verify.argtypes = [P, P, I64, ctypes.c_int32, P, P, P, P, I, I, P, P, P, P, SZ, P]
        L.irm_pages_workspace_size.argtypes = [I, P]
        L.irm_pages_resize.argtypes = [P, P, I, P, I, P, I64, P, SZ, P]
        L.irm_pages_fork.argtypes = [P, P, I, P, I, P, I, P, I, P, I64, P, SZ, P]
        L.irm_pages_compact.argtypes = [P, I, I64, P, I, I, P, P, I, P, P, SZ, P]
        L.irm_pages_copy.argtypes = [P, I, I64, P, P, I, P]
        for name in EXPORTS:
            if name not in ("irm_status_string", "irm_last_error", "irm_version"):
                getattr(L, name).restype = I
        _lib = L
    return _lib


def _check(st: int):
    if st != 0:
        L = lib()
        raise IrmError(st, L.irm_status_string(st).decode(), L.irm_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


class ChunkTable:
    """A batch of chunk tables in host memory, as the library takes them.  With CUDA present
    the table sits in one page-locked block laid out as the library's workspace table area
    (indptr [B+1] int32, padded to 8 bytes, then the chunk records), so a call stages it with
    one asynchronous host-to-device copy; keep it unchanged while calls that use it are in
    flight.  Without CUDA (host-only validation) it is plain pageable memory."""

    def __init__(self, chunks: np.ndarray, indptr: np.ndarray, pinned: bool | None = None):
        chunks = np.ascontiguousarray(chunks, dtype=CHUNK_DTYPE)
        indptr = np.ascontiguousarray(indptr, dtype=np.int32)
        self.B = int(indptr.shape[0] - 1)
        ia = (4 * (self.B + 1) + 7) // 8 * 8
        nbytes = ia + chunks.nbytes
        if pinned is None:
            pinned = torch.cuda.is_available()
        buf = torch.zeros(nbytes, dtype=torch.uint8)
        if pinned:
            buf = buf.pin_memory()
        self._buf = buf  # keeps the block alive
        raw = buf.numpy()
        self.indptr_host = raw[:4 * (self.B + 1)].view(np.int32)
        self.chunks_host = raw[ia:ia + chunks.nbytes].view(CHUNK_DTYPE)
        self.indptr_host[:] = indptr
        self.chunks_host[:] = chunks
        self.n_chunks = int(chunks.shape[0])

    def validate(self, n_rows: int) -> np.ndarray:
        ctx = np.zeros(self.B, np.int64)
        _check(lib().irm_validate_chunks(_ptr(self.chunks_host), _ptr(self.indptr_host), self.B,
                                         int(n_rows), _ptr(ctx)))
        return ctx


def validate_chunks(chunks: np.ndarray, indptr: np.ndarray, n_rows: int) -> np.ndarray:
    """Host-only validation (no GPU needed).  Returns each request's context length."""
    chunks = np.ascontiguousarray(chunks, dtype=CHUNK_DTYPE)
    indptr = np.ascontiguousarray(indptr, dtype=np.int32)
    B = int(indptr.shape[0] - 1)
    ctx = np.zeros(max(B, 1), np.int64)
    _check(lib().irm_validate_chunks(_ptr(chunks), _ptr(indptr), B, int(n_rows), _ptr(ctx)))
    return ctx[:B]


def new_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zero-initialised workspace (the first 256 bytes hold the device status word)."""
    return torch.zeros(max(int(nbytes), WORKSPACE_HEADER), dtype=torch.uint8, device=device)


def device_status(workspace: torch.Tensor, stream=None):
    """Raises IrmError if a kernel recorded a timeout or an out-of-range row (and clears it)."""
    _check(lib().irm_device_status(_ptr(workspace), _stream(stream)))


def selftest_wait_timeout(workspace: torch.Tensor, stream=None):
    """Launches the bounded-wait self-test (a wait nothing ever completes); after it,
    device_status(workspace) raises the timeout it recorded."""
    _check(lib().irm_selftest_wait_timeout(_ptr(workspace), workspace.numel(), _stream(stream)))


def assemble_kv_workspace_size(table: ChunkTable) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().irm_assemble_kv_workspace_size(_ptr(table.chunks_host), _ptr(table.indptr_host),
                                                table.B, ctypes.byref(n)))
    return n.value


def irm_assemble_kv(table: ChunkTable, kv_rows: torch.Tensor, paged_out=None, page_table=None,
                    out_src_row=None, out_delta=None, out_pos_src=None, workspace=None,
                    stream=None, rope: Rope | None = None):
    """Rotate+gather and/or the assembly plan; rope selects the model's RoPE variant
    (irm_assemble_kv_rope), None the default."""
    _need(kv_rows, torch.bfloat16, "kv_rows", 2)
    n_pages, max_pages = 0, 0
    if paged_out is not None:
        _need(paged_out, torch.bfloat16, "paged_out", 3)
        _need(page_table, torch.int32, "page_table", 2)
        n_pages, max_pages = int(paged_out.shape[0]), int(page_table.shape[1])
    for t, n in ((out_src_row, "out_src_row"), (out_delta, "out_delta"), (out_pos_src, "out_pos_src")):
        if t is not None:
            _need(t, torch.int32, n, 1)
    if workspace is None:
        workspace = new_workspace(assemble_kv_workspace_size(table), kv_rows.device)
    _check(lib().irm_assemble_kv_rope(
        _ptr(table.chunks_host), _ptr(table.indptr_host), table.B,
        _ptr(kv_rows), int(kv_rows.shape[0]), _ptr(paged_out), n_pages,
        _ptr(page_table), max_pages, _ptr(out_src_row), _ptr(out_delta), _ptr(out_pos_src),
        _rope_ptr(rope), _ptr(workspace), workspace.numel(), _stream(stream)))
    return workspace


def decode_workspace_size(table: ChunkTable, H: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().irm_mla_attn_decode_workspace_size(_ptr(table.chunks_host),
                                                    _ptr(table.indptr_host), table.B, int(H),
                                                    ctypes.byref(n)))
    return n.value


def prefill_workspace_size(table: ChunkTable, n_q: int, H: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().irm_mla_attn_prefill_workspace_size(_ptr(table.chunks_host), _ptr(table.indptr_host),
                                                     table.B, int(n_q), int(H), ctypes.byref(n)))
    return n.value


def irm_mla_attn_decode(q_lat, q_rope, table: ChunkTable, kv_rows, softmax_scale=DEFAULT_SCALE,
                        out=None, lse=None, workspace=None, stream=None, rope: Rope | None = None):
    """q_lat [B, H, 512] / q_rope [B, H, 64] bf16 (a [B, 1, H, *] view is accepted); rope
    selects the model's RoPE variant (irm_mla_attn_decode_rope), None the default."""
    B, H = int(q_lat.shape[0]), int(q_lat.shape[-2])
    _need(q_lat, torch.bfloat16, "q_lat")
    _need(q_rope, torch.bfloat16, "q_rope")
    _need(kv_rows, torch.bfloat16, "kv_rows", 2)
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q_lat.device)
    _need(out, torch.bfloat16, "out")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    if workspace is None:
        workspace = new_workspace(decode_workspace_size(table, H), q_lat.device)
    _check(lib().irm_mla_attn_decode_rope(
        _ptr(q_lat), _ptr(q_rope), B, H, _ptr(table.chunks_host), _ptr(table.indptr_host),
        _ptr(kv_rows), int(kv_rows.shape[0]),
        float(softmax_scale), _ptr(out), _ptr(lse), _rope_ptr(rope), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return out, lse, workspace


def irm_mla_attn_decode_noalloc(q_lat, q_rope, table: ChunkTable, kv_rows,
                                softmax_scale=DEFAULT_SCALE, out=None, lse=None, stream=None):
    """Decode for callers that cannot allocate device memory: the library's own fixed
    scratch array replaces the workspace (see include/irm.h for the limit)."""
    B, H = int(q_lat.shape[0]), int(q_lat.shape[-2])
    _need(q_lat, torch.bfloat16, "q_lat")
    _need(q_rope, torch.bfloat16, "q_rope")
    _need(kv_rows, torch.bfloat16, "kv_rows", 2)
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q_lat.device)
    _need(out, torch.bfloat16, "out")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    _check(lib().irm_mla_attn_decode_noalloc(
        _ptr(q_lat), _ptr(q_rope), B, H, _ptr(table.chunks_host), _ptr(table.indptr_host),
        _ptr(kv_rows), int(kv_rows.shape[0]),
        float(softmax_scale), _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


def decode_noalloc_status(stream=None):
    """Raises IrmError if a no-allocation decode recorded a timeout or an out-of-range row in
    the library's scratch array (and clears it)."""
    _check(lib().irm_decode_noalloc_status(_stream(stream)))


def irm_mla_attn_prefill(q_lat, q_rope, table: ChunkTable, kv_rows, softmax_scale=DEFAULT_SCALE,
                         out=None, lse=None, workspace=None, stream=None, rope: Rope | None = None):
    """q_lat [B, n_q, H, 512] / q_rope [B, n_q, H, 64] bf16, causal over the last n_q rows;
    rope selects the model's RoPE variant (irm_mla_attn_prefill_rope), None the default."""
    B, n_q, H = (int(x) for x in q_lat.shape[:3])
    _need(q_lat, torch.bfloat16, "q_lat", 4)
    _need(q_rope, torch.bfloat16, "q_rope", 4)
    _need(kv_rows, torch.bfloat16, "kv_rows", 2)
    if out is None:
        out = torch.empty((B, n_q, H, 512), dtype=torch.bfloat16, device=q_lat.device)
    _need(out, torch.bfloat16, "out")
    if lse is not None:
        _need(lse, torch.float32, "lse")
    if workspace is None:
        workspace = new_workspace(prefill_workspace_size(table, n_q, H), q_lat.device)
    _check(lib().irm_mla_attn_prefill_rope(
        _ptr(q_lat), _ptr(q_rope), B, n_q, H, _ptr(table.chunks_host), _ptr(table.indptr_host),
        _ptr(kv_rows), int(kv_rows.shape[0]),
        float(softmax_scale), _ptr(out), _ptr(lse), _rope_ptr(rope), _ptr(workspace),
        workspace.numel(), _stream(stream)))
    return out, lse, workspace


def cdc_sizes(offsets: np.ndarray, params: CdcParams | None = None):
    """(workspace bytes, output slots) of irm_cdc_chunk for these stream offsets."""
    offsets = np.ascontiguousarray(offsets, dtype=np.int64)
    nb, sl = ctypes.c_size_t(0), ctypes.c_int64(0)
    pp = None if params is None else ctypes.cast(ctypes.pointer(params), ctypes.c_void_p)
    _check(lib().irm_cdc_sizes(_ptr(offsets), int(offsets.shape[0] - 1), pp, ctypes.byref(nb),
                               ctypes.byref(sl)))
    return nb.value, sl.value


def cdc_slot_base(offsets: np.ndarray, min_len: int = 32) -> np.ndarray:
    """First output slot of each stream (the layout irm_cdc_sizes documents)."""
    lens = np.diff(np.asarray(offsets, np.int64))
    return np.concatenate([[0], np.cumsum(lens // min_len + 1)])[:-1]


def irm_cdc_chunk(tokens: torch.Tensor, offsets: np.ndarray, gear: torch.Tensor | None,
                  params: CdcParams | None = None, fingerprints=True, out=None, workspace=None,
                  stream=None, vocab: int | None = None):
    """Content-defined chunks of token streams (tokens int32 on the GPU, streams at host
    offsets; gear: the 64-bit Gear table as an int64 tensor on the GPU, or None for Gear
    words generated from params.gear_seed, with token ids in [0, vocab)).  Returns
    (n_chunks [S], chunk_start [slots], chunk_len [slots], chunk_hash [slots] or None,
    workspace); stream s's chunks sit at slots cdc_slot_base(offsets)[s] onwards."""
    _need(tokens, torch.int32, "tokens", 1)
    if gear is not None:
        _need(gear, torch.int64, "gear", 1)
        vocab = int(gear.shape[0])
    elif vocab is None:
        raise ValueError("generated Gear words need the vocab size")
    offsets = np.ascontiguousarray(offsets, dtype=np.int64)
    S = int(offsets.shape[0] - 1)
    nbytes, slots = cdc_sizes(offsets, params)
    dev = tokens.device
    if out is None:
        out = (torch.empty(S, dtype=torch.int32, device=dev),
               torch.empty(max(slots, 1), dtype=torch.int32, device=dev),
               torch.empty(max(slots, 1), dtype=torch.int32, device=dev),
               torch.empty(max(slots, 1), dtype=torch.int64, device=dev) if fingerprints else None)
    n_chunks, c_start, c_len, c_hash = out
    if workspace is None:
        workspace = new_workspace(nbytes, dev)
    pp = None if params is None else ctypes.cast(ctypes.pointer(params), ctypes.c_void_p)
    _check(lib().irm_cdc_chunk(_ptr(tokens), _ptr(offsets), S, _ptr(gear),
                               int(vocab), pp, _ptr(n_chunks), _ptr(c_start), _ptr(c_len),
                               _ptr(c_hash), _ptr(workspace), workspace.numel(), _stream(stream)))
    return n_chunks, c_start, c_len, c_hash, workspace


def _host_i32(x, name):
    if type(x) is np.ndarray and x.dtype == np.int32 and x.ndim == 1 and x.flags.c_contiguous:
        return x
    a = np.asarray(x)
    if a.ndim != 1 or a.dtype.kind not in "iu":
        raise ValueError(f"{name} must be a 1-d integer array in host memory")
    if a.itemsize >= 4 and a.size and (a.max() > 2**31 - 1 or a.min() < -2**31):
        raise ValueError(f"{name} has values outside int32")
    return np.ascontiguousarray(a, dtype=np.int32)


def _size(t, dim, name):
    """A size that a call takes from one of its tensors."""
    if not isinstance(t, torch.Tensor) or t.dim() <= dim:
        raise ValueError(f"{name} must be a tensor on the GPU with more than {dim} dimensions")
    return t.shape[dim]


def _take(t, dtype, shape, name, device):
    """Address of a contiguous GPU tensor of this type, shape and device (a call takes several, so one
    comparison each; what is wrong is only looked for when something is)."""
    if (type(t) is torch.Tensor and t.get_device() == device.index and t.dtype is dtype and t.shape == shape
            and t.is_cuda and t.is_contiguous()):
        return t.data_ptr()
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    return t.data_ptr()


def _make(new, device, stream):
    """new(): tensors that a call makes for itself, allocated (and zeroed) on the stream that the call runs on."""
    if stream is None:
        return new()
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on {device}")
    with torch.cuda.stream(stream):
        return new()


def _take_workspace(workspace, nbytes, device, stream):
    """(workspace, its address, its bytes); a new one of nbytes() where the caller keeps none."""
    if workspace is None:
        workspace = _make(lambda: new_workspace(nbytes(), device), device, stream)
    n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
    return workspace, _take(workspace, torch.uint8, (n,), "workspace", device), n


def _launch(fn, device, stream, *args):
    """A library call on `device` (made current for it) and on `stream`, by default the device's current one."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device.index)
    else:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the call's tensors on {device}")
        stream = stream.cuda_stream
    if device.index == torch._C._cuda_getDevice():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != 0:
        _check(st)


def tree_workspace_size(ctx: np.ndarray, q_indptr: np.ndarray, H: int) -> int:
    """Workspace bytes of irm_mla_attn_tree for these lengths."""
    ctx, q_indptr = _host_i32(ctx, "ctx"), _host_i32(q_indptr, "q_indptr")
    if len(q_indptr) != len(ctx) + 1:
        raise ValueError("q_indptr must have one entry more than ctx")
    n = ctypes.c_size_t(0)
    _check(lib().irm_mla_attn_tree_workspace_size(ctx.tobytes(), q_indptr.tobytes(), len(ctx), int(H), ctypes.byref(n)))
    return n.value


def irm_mla_attn_tree(q_lat, q_rope, ctx, q_indptr, paged_kv, page_table, tree_mask, softmax_scale=DEFAULT_SCALE,
                      out=None, lse=None, workspace=None, stream=None):
    """Attention of drafted trees over the paged cache: q_lat [T, H, 512] / q_rope [T, H, 64] bf16 of
    all nodes end to end, ctx [B] and q_indptr [B + 1] integers in host memory, paged_kv [n_pages, 64,
    576] bf16, page_table [B, max_pages] int32, tree_mask [T, words] int32 (bit k of a row: the node
    sees draft k).  Returns (out [T, H, 512] bf16, lse or None, workspace)."""
    ctx, q_indptr = _host_i32(ctx, "ctx"), _host_i32(q_indptr, "q_indptr")
    B = len(ctx)
    if B < 1 or len(q_indptr) != B + 1:
        raise ValueError("q_indptr must have one entry more than ctx")
    if not isinstance(q_lat, torch.Tensor) or q_lat.dim() != 3:
        _need(q_lat, torch.bfloat16, "q_lat", 3)
    dev, T, H = q_lat.device, int(q_indptr[B]), q_lat.shape[1]
    ql = _take(q_lat, torch.bfloat16, (T, H, 512), "q_lat", dev)
    n_pages, max_pages, words = _size(paged_kv, 0, "paged_kv"), _size(page_table, 1, "page_table"), _size(tree_mask, 1, "tree_mask")
    qr = _take(q_rope, torch.bfloat16, (T, H, 64), "q_rope", dev)
    kv = _take(paged_kv, torch.bfloat16, (n_pages, 64, 576), "paged_kv", dev)
    pt = _take(page_table, torch.int32, (B, max_pages), "page_table", dev)
    tm = _take(tree_mask, torch.int32, (T, words), "tree_mask", dev)
    if out is None:
        out = _make(lambda: torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev), dev, stream)
    o = _take(out, torch.bfloat16, (T, H, 512), "out", dev)
    ls = None if lse is None else _take(lse, torch.float32, (T, H), "lse", dev)
    workspace, ws, ws_bytes = _take_workspace(workspace, lambda: tree_workspace_size(ctx, q_indptr, H), dev, stream)
    if T > 0:
        _launch(lib().irm_mla_attn_tree, dev, stream, ql, qr, B, H, ctx.tobytes(), q_indptr.tobytes(), kv, n_pages, pt, max_pages,
                tm, words, softmax_scale, o, ls, ws, ws_bytes)
    return out, lse, workspace


def _take_probs(t, shape, name, device):
    """Address and row stride of fp32 rows that may lie in a wider buffer."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-d torch.float32 tensor on the GPU")
    if t.shape != shape or t.device != device:
        _take(t, torch.float32, shape, name, device)
    rows, vocab = shape
    ld = t.stride(0) if rows > 1 else vocab
    if ld < vocab or (vocab > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld


def irm_tree_verify(target_probs, tokens, parents, uniforms, q_indptr, draft_probs=None, max_path=None, out=None,
                    workspace=None, stream=None):
    """Verification of drafted trees: target_probs (and draft_probs) [T, vocab] fp32, rows may be
    strided; tokens, parents int32 [T], uniforms fp32 [T]; q_indptr [B + 1] integers in host
    memory.  Returns (n_accept [B], path [B, max_path], next_token [B], workspace), int32; max_path is
    the largest tree unless given (or taken from out, a tuple of the three)."""
    q_indptr = _host_i32(q_indptr, "q_indptr")
    B = len(q_indptr) - 1
    if B < 1:
        raise ValueError("q_indptr must have at least two entries")
    T = int(q_indptr[B])
    if not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 2:
        raise ValueError("target_probs must be a 2-d torch.float32 tensor on the GPU")
    dev, V = target_probs.device, target_probs.shape[1]
    tp, ld = _take_probs(target_probs, (T, V), "target_probs", dev)
    dp = None
    if draft_probs is not None:
        dp, draft_ld = _take_probs(draft_probs, (T, V), "draft_probs", dev)
        if draft_ld != ld:
            raise ValueError("draft_probs must have target_probs' row stride")
    tk = _take(tokens, torch.int32, (T,), "tokens", dev)
    pr = _take(parents, torch.int32, (T,), "parents", dev)
    un = _take(uniforms, torch.float32, (T,), "uniforms", dev)
    if out is None:
        if max_path is None:
            max_path = max(1, int((q_indptr[1:] - q_indptr[:-1]).max())) if B > 1 else max(1, T)
        out = _make(lambda: (torch.empty(B, dtype=torch.int32, device=dev),
                             torch.empty((B, max_path), dtype=torch.int32, device=dev),
                             torch.empty(B, dtype=torch.int32, device=dev)), dev, stream)
    n_accept, path, next_token = out
    if max_path is None:
        max_path = path.shape[1]
    na = _take(n_accept, torch.int32, (B,), "n_accept", dev)
    pa = _take(path, torch.int32, (B, max_path), "path", dev)
    nt = _take(next_token, torch.int32, (B,), "next_token", dev)
    workspace, ws, ws_bytes = _take_workspace(workspace, lambda: WORKSPACE_HEADER, dev, stream)
    _launch(lib().irm_tree_verify, dev, stream, tp, dp, ld, V, tk, pr, un, q_indptr.tobytes(), B, max_path, na, pa, nt, ws,
            ws_bytes)
    return n_accept, path, next_token, workspace


def pages_workspace_size(n_slots: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().irm_pages_workspace_size(int(n_slots), ctypes.byref(n)))
    return n.value


def _take_pages(seq_len, page_table, refcount):
    """Addresses and sizes of the page state: (device, n_slots, max_pages, n_pages, seq_len, page_table, refcount)."""
    n_slots, max_pages, n_pages = _size(seq_len, 0, "seq_len"), _size(page_table, 1, "page_table"), _size(refcount, 0, "refcount")
    dev = seq_len.device
    return (dev, n_slots, max_pages, n_pages, _take(seq_len, torch.int32, (n_slots,), "seq_len", dev),
            _take(page_table, torch.int32, (n_slots, max_pages), "page_table", dev),
            _take(refcount, torch.int32, (n_pages,), "refcount", dev))


def _take_cache(kv, device, n_pages=None):
    """[n_layers, n_pages, 64, 576] bf16, or one layer's [n_pages, 64, 576]: (address, layers, pages)."""
    if not isinstance(kv, torch.Tensor) or kv.dim() not in (3, 4):
        raise ValueError("kv must be [n_layers, n_pages, 64, 576] or [n_pages, 64, 576]")
    shape = kv.shape
    pages = shape[-3] if n_pages is None else n_pages
    layers = shape[0] if len(shape) == 4 else 1
    want = (layers, pages, 64, 576) if len(shape) == 4 else (pages, 64, 576)
    return _take(kv, torch.bfloat16, want, "kv", device), layers, pages


def irm_pages_resize(new_len, seq_len, page_table, refcount, workspace=None, stream=None):
    """Every request to new_len [n_slots] rows (device int32): allocates, trims or, with 0, frees its pages.
    seq_len [n_slots], page_table [n_slots, max_pages] and refcount [n_pages] (int32) are updated."""
    dev, n_slots, max_pages, n_pages, sl, pt, rc = _take_pages(seq_len, page_table, refcount)
    nl = _take(new_len, torch.int32, (n_slots,), "new_len", dev)
    workspace, ws, ws_bytes = _take_workspace(workspace, lambda: pages_workspace_size(n_slots), dev, stream)
    _launch(lib().irm_pages_resize, dev, stream, nl, sl, n_slots, pt, max_pages, rc, n_pages, ws, ws_bytes)
    return workspace


def irm_pages_fork(src, dst, kv, seq_len, page_table, refcount, workspace=None, stream=None):
    """Forks requests src into the empty slots dst (integers in host memory): full pages are shared, the
    partly filled last page is copied in every layer of kv ([n_layers, n_pages, 64, 576] bf16)."""
    src, dst = _host_i32(src, "src"), _host_i32(dst, "dst")
    if len(src) != len(dst):
        raise ValueError("src and dst must have the same length")
    dev, n_slots, max_pages, n_pages, sl, pt, rc = _take_pages(seq_len, page_table, refcount)
    cache, layers, _ = _take_cache(kv, dev, n_pages)
    workspace, ws, ws_bytes = _take_workspace(workspace, lambda: pages_workspace_size(n_slots), dev, stream)
    _launch(lib().irm_pages_fork, dev, stream, src.tobytes(), dst.tobytes(), len(src), cache, layers, sl, n_slots, pt, max_pages,
            rc, n_pages, ws, ws_bytes)
    return workspace


def irm_pages_compact(kv, page_table, base, path, n_accept, workspace=None, stream=None):
    """Moves accepted drafts' rows base + path[:, k] to base + k, k < n_accept, in every layer of kv; base,
    n_accept [n_slots] and path [n_slots, max_path] int32 on the device (irm_tree_verify's outputs)."""
    max_pages, max_path = _size(page_table, 1, "page_table"), _size(path, 1, "path")
    dev, n_slots = page_table.device, page_table.shape[0]
    cache, layers, n_pages = _take_cache(kv, dev)
    pt = _take(page_table, torch.int32, (n_slots, max_pages), "page_table", dev)
    ba = _take(base, torch.int32, (n_slots,), "base", dev)
    pa = _take(path, torch.int32, (n_slots, max_path), "path", dev)
    na = _take(n_accept, torch.int32, (n_slots,), "n_accept", dev)
    workspace, ws, ws_bytes = _take_workspace(workspace, lambda: WORKSPACE_HEADER, dev, stream)
    _launch(lib().irm_pages_compact, dev, stream, cache, layers, n_pages, pt, max_pages, n_slots, ba, pa, max_path, na, ws,
            ws_bytes)
    return workspace


def irm_pages_copy(kv, src, dst, stream=None):
    """Copies pages src[i] -> dst[i] (integers in host memory) in every layer of kv."""
    src, dst = _host_i32(src, "src"), _host_i32(dst, "dst")
    if len(src) != len(dst):
        raise ValueError("src and dst must have the same length")
    if not isinstance(kv, torch.Tensor):
        raise ValueError("kv must be [n_layers, n_pages, 64, 576] or [n_pages, 64, 576]")
    cache, layers, n_pages = _take_cache(kv, kv.device)
    _launch(lib().irm_pages_copy, kv.device, stream, cache, layers, n_pages, src.tobytes(), dst.tobytes(), len(src))


ASSEMBLE_S1 = 1


class Registry:
    """Content-addressed chunk registry (host side, libirm's irm_registry): keeps cached chunks'
    rows in a ring of pool rows and turns a request's CDC segments into a chunk table."""

    def __init__(self, pool_rows: int, pool_base: int = 0, capacity: int = 1 << 16):
        h = ctypes.c_void_p()
        _check(lib().irm_registry_create(int(pool_base), int(pool_rows), int(capacity), ctypes.byref(h)))
        self._h = h

    def close(self):
        if self._h:
            lib().irm_registry_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self):
        live, rows = ctypes.c_int64(0), ctypes.c_int64(0)
        _check(lib().irm_registry_stats(self._h, ctypes.byref(live), ctypes.byref(rows)))
        return live.value, rows.value

    def assemble(self, tokens, prefix_len, prefix_row, seg_start, seg_len, seg_hash, s1=False,
                 seed=0):
        """(chunk table as a CHUNK_DTYPE array, prefill flags uint8) of one request."""
        tokens = np.ascontiguousarray(tokens, dtype=np.int32)
        st = np.ascontiguousarray(seg_start, dtype=np.int32)
        ln = np.ascontiguousarray(seg_len, dtype=np.int32)
        hs = np.ascontiguousarray(np.asarray(seg_hash, dtype=np.uint64))
        cap = 1 + (int(((ln.astype(np.int64) + 127) // 128).sum()) if s1 else len(ln))
        out = np.zeros(cap, CHUNK_DTYPE)
        pre = np.zeros(cap, np.uint8)
        n = ctypes.c_int32(0)
        _check(lib().irm_registry_assemble(self._h, _ptr(tokens), int(tokens.shape[0]), int(prefix_len),
                                           int(prefix_row), _ptr(st), _ptr(ln), _ptr(hs), int(len(st)),
                                           ASSEMBLE_S1 if s1 else 0, ctypes.c_uint64(seed), _ptr(out),
                                           _ptr(pre), cap, ctypes.byref(n)))
        return out[:n.value], pre[:n.value]
