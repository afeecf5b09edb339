"""ctypes binding of libtq.so: the C ABI of include/tq.h under the same names.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI. Tensors must be CUDA tensors of the current device
(or of the device given by the first tensor argument, which is made current
for the call); sizes are passed through unchanged, and the library's status
codes become TQError. There is no CPU fallback: if libtq.so is missing the
first call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libtq.so")
CALL_PATH = os.path.join(_HERE, "_lib", "_tq_call.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "tq.h")

TQ_OK = 0
TQ_ERR_SHAPE = -1
TQ_ERR_NULL = -2
TQ_ERR_ALIGN = -3
TQ_ERR_CUDA = -4
TQ_ERR_TIMEOUT = -5
TQ_ERR_ALIAS = -6
TQ_ERR_WORKSPACE = -7
TQ_ERR_INDEX = -8
TQ_ERR_TYPE = -9

QK_K = 256
GROUP = 128
PQ2_0_BYTES = 34
PTQ1_0_BYTES = 28
Q8K_BYTES = 292
TILE_ROWS = 32
TILE_BYTES = 1088
STATIC_WS_BYTES = 8 << 20   # TQ_STATIC_WS_BYTES: fixed workspace of tq_matmul_static_ws

TQ_F32, TQ_F16, TQ_BF16 = 0, 1, 2
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_RAMP, ROPE_BANDS = range(5)

_lock = threading.Lock()
_lib = None


class TQError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        lib = _load()
        msg = lib.tq_strerror(code).decode()
        if code == TQ_ERR_CUDA:
            msg += f" (cudaError {lib.tq_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{code}]")


def header_functions() -> list[str]:
    """Names of the functions include/tq.h declares."""
    with open(HEADER) as f:
        src = f.read()
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(tq_\w+)\s*\(", src, flags=re.M)


def _load():
    global _lib
    if _lib is not None:   # loaded: no lock on the per-call path
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build the CUDA library first "
                "(python -m bit_matvec_gb300.build, or __graft_entry__.build())")
        lib = ctypes.CDLL(LIB_PATH)
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        F, D = ctypes.c_float, ctypes.c_double
        sig = {
            "tq_quantize_q8K": ([P, P, I64, I64, P], I),
            "tq_repacked_bytes": ([I64, I64], I64),
            "tq_repack": ([P, P, I64, I64, P], I),
            "tq_unrepack": ([P, P, I64, I64, P], I),
            "tq_ptq1_0_bytes": ([I64, I64], I64),
            "tq_repack_ptq1_0": ([P, P, I64, I64, P], I),
            "tq_matmul": ([P, P, P, I64, I64, I64, P], I),
            "tq_matmul_groupsums": ([P, P, P, I64, I64, I64, P], I),
            "tq_matmul_workspace_bytes": ([I64, I64, I64], I64),
            "tq_matmul_ws": ([P, P, P, I64, I64, I64, P, I64, P], I),
            "tq_matmul_groupsums_ws": ([P, P, P, I64, I64, I64, P, I64, P], I),
            "tq_matmul_static_ws": ([P, P, P, I64, I64, I64, P], I),
            "tq_matmul_host": ([P, P, P, P, P, P, I64, I64, I64, P, I64, P], I),
            "tq_quantize_matmul": ([P, P, P, P, I64, I64, I64, P, I64, P], I),
            "tq_strerror": ([I], ctypes.c_char_p),
            "tq_last_cuda_error": ([], I),
            "tq_device_status": ([], I),
            "tq_version": ([], ctypes.c_char_p),
            "tq_debug_stall_next_launch": ([I64], I),
            "tq_probe_read_sum": ([P, I64, P, I, P], I),
            "tq_ptq1_0_stream_bytes": ([I64, I64], I64),
            "tq_repack_ptq1_0_stream": ([P, P, I64, I64, P], I),
            "tq_matmul_ptq1_0_stream": ([P, P, P, I64, I64, I64, P], I),
            "tq_matmul_ptq1_0_stream_groupsums": ([P, P, P, I64, I64, I64, P], I),
            "tq_rope_turns": ([I64, D, I, D, D, D, D, P, P], I),
            "tq_qk_norm_rope": ([P, I64, P, I64, I, P, I64, P, I64, I, I64, I64, I64, I64, P, P,
                                 F, P, P, P], I),
            "tq_kv_append": ([P, I64, P, I64, P, I64, I, P, I64, P, P, P, I64, I64, P, P, F, P,
                              P], I),
            "tq_paged_attention": ([P, I64, P, P, P, P, I64, I, P, I64, I64, I64, I64, F, I64, P,
                                    I64, P], I),
            "tq_paged_attention_workspace_bytes": ([I64] * 8, I64),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def library() -> ctypes.CDLL:
    """The loaded libtq.so (raises if it has not been built)."""
    return _load()


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()   # an int; the declared argtypes make it a void*


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _call(name, device, *args):
    lib = _load()
    if device.index is None or device.index == torch.cuda.current_device():
        rc = getattr(lib, name)(*args)
    else:
        with torch.cuda.device(device):
            rc = getattr(lib, name)(*args)
    if rc != TQ_OK:
        raise TQError(rc, name)


# ---------------------------------------------------------------- allocation helpers

def q8K_nbytes(ntok: int, cols: int) -> int:
    return ntok * (cols // QK_K) * Q8K_BYTES


def q8K_empty(ntok: int, cols: int, device="cuda") -> torch.Tensor:
    """uint8 buffer for ntok x cols/256 q8_K blocks."""
    return torch.empty(q8K_nbytes(ntok, cols), dtype=torch.uint8, device=device)


def tq_repacked_bytes(rows: int, cols: int) -> int:
    n = _load().tq_repacked_bytes(rows, cols)
    if n < 0:
        raise TQError(TQ_ERR_SHAPE, "tq_repacked_bytes")
    return int(n)


def repacked_empty(rows: int, cols: int, device="cuda") -> torch.Tensor:
    return torch.empty(tq_repacked_bytes(rows, cols), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- the C ABI

def tq_quantize_q8K(X: torch.Tensor, Xq: torch.Tensor, ntok: int, cols: int, stream=None):
    _call("tq_quantize_q8K", X.device, _ptr(X), _ptr(Xq), ntok, cols, _stream(stream, X.device))


def tq_repack(Wpq2: torch.Tensor, Wtq: torch.Tensor, rows: int, cols: int, stream=None):
    _call("tq_repack", Wpq2.device, _ptr(Wpq2), _ptr(Wtq), rows, cols,
          _stream(stream, Wpq2.device))


def tq_unrepack(Wtq: torch.Tensor, Wpq2: torch.Tensor, rows: int, cols: int, stream=None):
    _call("tq_unrepack", Wtq.device, _ptr(Wtq), _ptr(Wpq2), rows, cols,
          _stream(stream, Wtq.device))


def tq_ptq1_0_bytes(rows: int, cols: int) -> int:
    n = _load().tq_ptq1_0_bytes(rows, cols)
    if n < 0:
        raise TQError(TQ_ERR_SHAPE, "tq_ptq1_0_bytes")
    return int(n)


def tq_repack_ptq1_0(Wpt: torch.Tensor, Wtq: torch.Tensor, rows: int, cols: int, stream=None):
    """ptq1_0 (1.75-bit) weights -> the tq layout, decoded once at load."""
    _call("tq_repack_ptq1_0", Wpt.device, _ptr(Wpt), _ptr(Wtq), rows, cols,
          _stream(stream, Wpt.device))


def tq_ptq1_0_stream_bytes(rows: int, cols: int) -> int:
    n = _load().tq_ptq1_0_stream_bytes(rows, cols)
    if n < 0:
        raise TQError(TQ_ERR_SHAPE, "tq_ptq1_0_stream_bytes")
    return int(n)


def tq_repack_ptq1_0_stream(Wpt: torch.Tensor, Wt1: torch.Tensor, rows: int, cols: int,
                            stream=None):
    """ptq1_0 (1.75-bit) weights -> 32-row stream tiles, not decoded."""
    _call("tq_repack_ptq1_0_stream", Wpt.device, _ptr(Wpt), _ptr(Wt1), rows, cols,
          _stream(stream, Wpt.device))


def tq_matmul_ptq1_0_stream(Wt1: torch.Tensor, Xq: torch.Tensor, Y: torch.Tensor, rows: int,
                            cols: int, ntok: int, stream=None):
    _call("tq_matmul_ptq1_0_stream", Wt1.device, _ptr(Wt1), _ptr(Xq), _ptr(Y), rows, cols, ntok,
          _stream(stream, Wt1.device))


def tq_matmul_ptq1_0_stream_groupsums(Wt1: torch.Tensor, Xq: torch.Tensor, S: torch.Tensor,
                                      rows: int, cols: int, ntok: int, stream=None):
    _call("tq_matmul_ptq1_0_stream_groupsums", Wt1.device, _ptr(Wt1), _ptr(Xq), _ptr(S), rows,
          cols, ntok, _stream(stream, Wt1.device))


def tq_matmul(Wtq: torch.Tensor, Xq: torch.Tensor, Y: torch.Tensor, rows: int, cols: int,
              ntok: int, stream=None):
    _call("tq_matmul", Wtq.device, _ptr(Wtq), _ptr(Xq), _ptr(Y), rows, cols, ntok,
          _stream(stream, Wtq.device))


def tq_matmul_groupsums(Wtq: torch.Tensor, Xq: torch.Tensor, S: torch.Tensor, rows: int,
                        cols: int, ntok: int, stream=None):
    _call("tq_matmul_groupsums", Wtq.device, _ptr(Wtq), _ptr(Xq), _ptr(S), rows, cols, ntok,
          _stream(stream, Wtq.device))


def tq_matmul_workspace_bytes(rows: int, cols: int, ntok: int) -> int:
    n = _load().tq_matmul_workspace_bytes(rows, cols, ntok)
    if n < 0:
        raise TQError(TQ_ERR_SHAPE, "tq_matmul_workspace_bytes")
    return int(n)


def workspace_empty(rows: int, cols: int, ntok: int, device="cuda") -> torch.Tensor:
    """uint8 buffer for tq_matmul_ws (at least one byte, so it has an address)."""
    return torch.empty(max(1, tq_matmul_workspace_bytes(rows, cols, ntok)), dtype=torch.uint8,
                       device=device)


def tq_matmul_ws(Wtq: torch.Tensor, Xq: torch.Tensor, Y: torch.Tensor, rows: int, cols: int,
                 ntok: int, workspace: torch.Tensor, stream=None):
    _call("tq_matmul_ws", Wtq.device, _ptr(Wtq), _ptr(Xq), _ptr(Y), rows, cols, ntok,
          _ptr(workspace), workspace.numel(), _stream(stream, Wtq.device))


def tq_matmul_groupsums_ws(Wtq: torch.Tensor, Xq: torch.Tensor, S: torch.Tensor, rows: int,
                           cols: int, ntok: int, workspace: torch.Tensor, stream=None):
    _call("tq_matmul_groupsums_ws", Wtq.device, _ptr(Wtq), _ptr(Xq), _ptr(S), rows, cols, ntok,
          _ptr(workspace), workspace.numel(), _stream(stream, Wtq.device))


def tq_matmul_static_ws(Wtq: torch.Tensor, Xq: torch.Tensor, Y: torch.Tensor, rows: int,
                        cols: int, ntok: int, stream=None):
    """tq_matmul_ws with the library's fixed STATIC_WS_BYTES device array as
    its workspace, for callers that cannot allocate device memory. Calls share
    that array: calls that overlap on the GPU race, so keep them ordered."""
    _call("tq_matmul_static_ws", Wtq.device, _ptr(Wtq), _ptr(Xq), _ptr(Y), rows, cols, ntok,
          _stream(stream, Wtq.device))


def tq_quantize_matmul(Wtq: torch.Tensor, X: torch.Tensor, Xq: torch.Tensor, Y: torch.Tensor,
                       rows: int, cols: int, ntok: int, workspace: torch.Tensor, stream=None):
    """Xq = q8_K(X) and Y = Wtq x Xq in one call (one fused launch up to 3 tokens; from 4 to
    8, where the workspace size is not 0, a staging kernel and the GEMV)."""
    _call("tq_quantize_matmul", Wtq.device, _ptr(Wtq), _ptr(X), _ptr(Xq), _ptr(Y), rows, cols,
          ntok, _ptr(workspace), workspace.numel(), _stream(stream, Wtq.device))


def _host_ptr(t: torch.Tensor):
    if t.is_cuda:
        raise ValueError("tensor must live in host memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def tq_matmul_host(Wtq: torch.Tensor, X_host: torch.Tensor, X: torch.Tensor, Xq: torch.Tensor,
                   Y: torch.Tensor, Y_host: torch.Tensor, rows: int, cols: int, ntok: int,
                   workspace: torch.Tensor, stream=None):
    """Host f32 activations in, host f32 outputs out, in one enqueued step (copy
    in, quantize, matmul, copy out); X_host and Y_host should be pinned. Returns
    at once: synchronize the stream before reading Y_host."""
    _call("tq_matmul_host", Wtq.device, _ptr(Wtq), _host_ptr(X_host), _ptr(X), _ptr(Xq), _ptr(Y),
          _host_ptr(Y_host), rows, cols, ntok, _ptr(workspace), workspace.numel(),
          _stream(stream, Wtq.device))


# ---------------------------------------------------------------- norm, rotation, cache, attention

_TYPES = {torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16}

# The calls below run for a few microseconds on the GPU for a few tokens, so their arguments are
# marshalled in C (csrc/tq_call.c).

_call_module = None
_OTHER_DEVICE = 1   # what its functions return when the tensors are not on the current device


def _calls():
    global _call_module
    if _call_module is None:
        lib = _load()
        if not os.path.exists(CALL_PATH):
            raise RuntimeError(f"{CALL_PATH} is missing: build the library first "
                               "(python -m bit_matvec_gb300.build, or __graft_entry__.build())")
        loader = importlib.machinery.ExtensionFileLoader("_tq_call", CALL_PATH)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location("_tq_call", CALL_PATH, loader=loader))
        loader.exec_module(module)
        module.setup((torch.float32, torch.float16, torch.bfloat16, torch.int32),
                     torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream,
                     tuple(ctypes.cast(f, ctypes.c_void_p).value for f in
                           (lib.tq_qk_norm_rope, lib.tq_kv_append, lib.tq_paged_attention)))
        _call_module = module
    return _call_module


def _finish(rc: int, where: str, tensor: torch.Tensor, fn, args):
    """What a call's status asks for: the same again on the tensors' own device, or an exception."""
    if rc == _OTHER_DEVICE:
        with torch.cuda.device(tensor.device):
            rc = fn(*args)
    if rc != TQ_OK:
        raise TQError(rc, where)


def _type(t: torch.Tensor) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TQError(TQ_ERR_TYPE, str(t.dtype))
    return code


class Rope:
    """A rotation for tq_qk_norm_rope and tq_kv_append: turns is an int64 CUDA tensor of the
    rot_dim/2 entries tq_rope_turns gives (the bits of its unsigned fractions)."""

    class _Struct(ctypes.Structure):
        _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int64),
                    ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_float)]

    def __init__(self, turns: torch.Tensor, interleaved: bool = False, amplitude: float = 1.0):
        self.turns = turns   # kept alive: the struct holds its address
        if turns.dtype != torch.int64:
            raise ValueError("turns must be torch.int64")
        self.struct = Rope._Struct(_ptr(turns), 2 * turns.numel(), 1 if interleaved else 0,
                                   amplitude)
        self.ref = ctypes.addressof(self.struct)


class PagedKV:
    """A paged key/value cache: k and v of shape [pages][heads][page_size][head_dim], of any strides
    but a unit last one (a [pages][page_size][heads][head_dim] cache is passed transposed), and
    block_table int32 [sequences][pages of a sequence], whose rows may be longer than they are
    wide here. The tensors are used in place: update block_table and the cache freely between
    calls."""

    class _Struct(ctypes.Structure):
        _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                    ("block_table", ctypes.c_void_p)] + [
                        (n, ctypes.c_int64) for n in
                        ("nseq", "table_width", "table_stride", "pages", "page_size", "heads",
                         "head_dim", "page_stride", "head_stride", "slot_stride")] + [
                        ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor):
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.dim() != 4:
            raise ValueError("k and v must be alike: [pages][heads][page_size][head_dim]")
        if not (k.is_cuda and v.is_cuda and block_table.is_cuda):
            raise ValueError("tensor must live on a CUDA device")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("the last dimension must be contiguous")
        if block_table.dtype != torch.int32 or block_table.dim() != 2 or (
                block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError("block_table must be int32 [sequences][pages] with contiguous rows")
        self.k, self.v, self.block_table = k, v, block_table
        nseq, width = block_table.shape
        pages, heads, page_size, dim = k.shape
        self.struct = PagedKV._Struct(
            k.data_ptr(), v.data_ptr(), block_table.data_ptr(), nseq, width,
            block_table.stride(0) if nseq > 1 else width, pages, page_size, heads, dim,
            k.stride(0), k.stride(1), k.stride(2), _type(k), 0)
        self.ref = ctypes.addressof(self.struct)


def tq_rope_turns(rot_dim: int, base: float, kind: int = ROPE_PLAIN, factor: float = 1.0,
                  original_len: float = 0.0, low: float = 1.0, high: float = 32.0):
    """(turns, amplitude): the int64 CPU tensor that Rope takes (moved to the GPU), for a plain or a
    long-context rotation."""
    turns = torch.zeros(max(rot_dim, 0) // 2, dtype=torch.int64)
    amplitude = ctypes.c_float()
    rc = _load().tq_rope_turns(rot_dim, base, kind, factor, original_len, low, high,
                               turns.data_ptr(), ctypes.addressof(amplitude))
    if rc != TQ_OK:
        raise TQError(rc, "tq_rope_turns")
    return turns, amplitude.value


def tq_qk_norm_rope(Xq, Xk, Yq, Yk, positions=None, rope: Rope | None = None, q_weight=None,
                    k_weight=None, eps: float = 1e-6, stream=None):
    """Norm and rotation of the heads of Xq and Xk [tokens][heads][head_dim] (views of a fused
    projection's rows are fine) into Yq and Yk; Xk and Yk may be None."""
    fn = (_call_module or _calls()).qk_norm_rope
    args = (Xq, Xk, Yq, Yk, positions, None if rope is None else rope.ref, q_weight, k_weight, eps,
            stream)
    rc = fn(*args)
    if rc:
        _finish(rc, "tq_qk_norm_rope", Xq, fn, args)


def tq_kv_append(Xq, Xk, Xv, Yq, kv: PagedKV, seq_ids, positions, rope: Rope | None = None,
                 q_weight=None, k_weight=None, eps: float = 1e-6, stream=None):
    """The same, with the keys and the values Xv written to kv at positions[t] of sequence
    seq_ids[t]; Yq is of the cache's type. Xq and Yq may be None."""
    fn = (_call_module or _calls()).kv_append
    args = (Xq, Xk, Xv, Yq, kv.ref, seq_ids, positions, None if rope is None else rope.ref, q_weight,
            k_weight, eps, stream)
    rc = fn(*args)
    if rc:
        _finish(rc, "tq_kv_append", Xk, fn, args)


def tq_paged_attention_workspace_bytes(nseq: int, ntok: int, q_heads: int, kv_heads: int,
                                       head_dim: int, max_q: int, max_kv: int,
                                       window: int = 0) -> int:
    n = _load().tq_paged_attention_workspace_bytes(nseq, ntok, q_heads, kv_heads, head_dim, max_q,
                                                   max_kv, window)
    if n < 0:
        raise TQError(TQ_ERR_SHAPE, "tq_paged_attention_workspace_bytes")
    return int(n)


def tq_paged_attention(Q, kv: PagedKV, q_start, kv_len, O, max_q: int, max_kv: int, scale: float,
                       workspace=None, window: int = 0, lse=None, stream=None):
    """Causal attention of the new tokens Q [tokens][q_heads][head_dim], those of sequence b at
    q_start[b] .. q_start[b+1] - 1 and last of its kv_len[b] positions, over kv; O of any type."""
    fn = (_call_module or _calls()).paged_attention
    args = (Q, kv.ref, q_start, kv_len, O, max_q, max_kv, scale, workspace, window, lse, stream)
    rc = fn(*args)
    if rc:
        _finish(rc, "tq_paged_attention", Q, fn, args)


def tq_strerror(code: int) -> str:
    return _load().tq_strerror(code).decode()


def tq_last_cuda_error() -> int:
    return int(_load().tq_last_cuda_error())


def tq_device_status(device=None) -> int:
    """Read and clear the device status word (synchronizes the device)."""
    lib = _load()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return int(lib.tq_device_status())


def tq_probe_read_sum(buf: torch.Tensor, out: torch.Tensor, early: bool = False, stream=None):
    """Adds buf's 32-bit words (mod 2^32) to out[0] (an int32 tensor) with the
    read-ceiling probe kernel: one streaming pass over buf and nothing else."""
    _call("tq_probe_read_sum", buf.device, _ptr(buf), buf.numel() * buf.element_size(), _ptr(out),
          1 if early else 0, _stream(stream, buf.device))


def tq_debug_stall_next_launch(wait_limit_ns: int):
    """Test facility: the next matmul kernel's first thread block requests no
    input copies, so its waits expire after wait_limit_ns and it reports
    TQ_ERR_TIMEOUT through tq_device_status (0 cancels)."""
    rc = _load().tq_debug_stall_next_launch(wait_limit_ns)
    if rc != TQ_OK:
        raise TQError(rc, "tq_debug_stall_next_launch")


def tq_version() -> str:
    return _load().tq_version().decode()
