"""grouped_expert_gemm_amd — Python binding of libgeg (grouped 4-bit expert GEMM, gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in include/geg.h. torch supplies device
memory and the current stream. There is no CPU fallback: host tensors are
refused, and a missing library raises.

    out = gnf4_grouped_gemm(a, sizes, w, absmax)          # NF4 forward
    out = gmxfp4_grouped_gemm(a, sizes, blocks, scales)   # MXFP4 forward
    dx  = gnf4_grouped_dgrad(dy, sizes, w, absmax)        # NF4 input gradient
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading

__all__ = [
    "GegError", "GegDeviceError", "Opts", "Workspace", "lib", "header_functions",
    "gnf4_grouped_gemm", "gnf4_grouped_gemm_noalloc", "gmxfp4_grouped_gemm", "gnf4_grouped_dgrad", "gmxfp4_grouped_dgrad",
    "grouped_linear", "gnf4_expert_block", "gmxfp4_expert_block", "route_sort", "route_combine",
    "gnf4_dequant", "gmxfp4_dequant", "gnf4_quantize", "geg_workspace_bytes",
    "gmxfp4_w4a8_grouped_gemm", "gmxfp8_quantize", "GEG_OP_MXFP4_W4A8", "DEVERR_NON_FINITE",
    "gnf4_grouped_gemm_lora", "gmxfp4_grouped_gemm_lora", "gnf4_grouped_dgrad_lora",
    "gmxfp4_grouped_dgrad_lora", "grouped_linear_lora",
    "geg_version", "geg_launch_count", "GEG_OP_NF4_FWD", "GEG_OP_MXFP4_FWD", "GEG_OP_NF4_DGRAD",
    "GEG_OP_NF4_BLOCK", "GEG_OP_MXFP4_BLOCK", "GEG_OP_MXFP4_DGRAD", "DEVERR_NEGATIVE_SIZE", "DEVERR_SIZES_EXCEED_M", "DEVERR_FP16_RANGE",
    "DEVERR_BAD_EXPERT_ID",
    "gmxfp4_quantize", "gmxfp4_w4a4_grouped_gemm", "GEG_OP_MXFP4_W4A4", "route_topk", "route_topk_grad", "route_combine_grad",
    "gnf4_moe_layer", "gmxfp4_moe_layer", "router_gate", "dispatch_rows", "combine_rows",
    "grouped_gemm", "grouped_dgrad", "grouped_wgrad", "grouped_matmul", "request_lora",
    "philox_dropout", "dropout",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgeg.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "geg.h")

GEG_OP_NF4_FWD, GEG_OP_MXFP4_FWD, GEG_OP_NF4_DGRAD = 0, 1, 2
GEG_OP_NF4_BLOCK, GEG_OP_MXFP4_BLOCK, GEG_OP_MXFP4_DGRAD = 3, 4, 5
GEG_OP_MXFP4_W4A8 = 6
GEG_OP_MXFP4_W4A4 = 8
DEVERR_NEGATIVE_SIZE, DEVERR_SIZES_EXCEED_M, DEVERR_FP16_RANGE = 0x1, 0x2, 0x4
DEVERR_BAD_EXPERT_ID, DEVERR_NON_FINITE = 0x8, 0x10

_STATUS = {0: "GEG_OK", 1: "GEG_ERR_NULL_POINTER", 2: "GEG_ERR_BAD_SHAPE", 3: "GEG_ERR_MISALIGNED",
           4: "GEG_ERR_NOT_DEVICE_MEMORY", 5: "GEG_ERR_WORKSPACE", 6: "GEG_ERR_UNSUPPORTED_DEVICE",
           7: "GEG_ERR_HIP", 8: "GEG_ERR_BAD_OPTION", 9: "device error word"}


class GegError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_STATUS.get(status, status)}: {detail}")


class Opts(ctypes.Structure):
    """geg_opts: force_path 0 auto / 1 skinny / 2 tiled / 3 vector / 4 narrow; split_k 0
    or 1 none / 2..16 (skinny); kernel_events: NULL or a pointer to 4 hipEvent_t (tile start/end,
    decode start/end) recorded around the call's kernels; cu_limit 0, or n > 0 to size every
    grid for at most n compute units (persistent loops then run more rounds; for tests)."""
    _fields_ = [("force_path", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("kernel_events", ctypes.c_void_p), ("cu_limit", ctypes.c_int32)]


class GegDeviceError(GegError):
    """A call's kernels flagged a condition in the workspace's device error word
    (GEG_DEVERR_* bits): raised by the wrappers when called with check_errors=True."""

    NAMES = {0x1: "negative sizes[e] (treated as 0)", 0x2: "sum(sizes) > M (rows past M not computed)",
             0x4: "an fp16 operand overflowed or is not finite", 0x8: "a top-k id outside [0, E) (dropped)",
             0x10: "a non-finite W4A8 activation"}

    def __init__(self, bits: int):
        self.bits = bits
        what = "; ".join(v for k, v in self.NAMES.items() if bits & k) or "unknown bits"
        super().__init__(9, f"device error word 0x{bits:x}: {what}")


_lib = None
_lib_lock = threading.Lock()
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load libgeg.so (built in-tree by grouped_expert_gemm_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build it with `python -m grouped_expert_gemm_amd.build` "
                    "(hipcc, gfx950). There is no fallback implementation.")
            L = ctypes.CDLL(LIB_PATH)
            gemm_args = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P, _P]
            for name in ("gnf4_grouped_gemm", "gmxfp4_grouped_gemm", "gnf4_grouped_dgrad",
                         "gmxfp4_grouped_dgrad", "gmxfp4_w4a8_grouped_gemm", "gmxfp4_w4a4_grouped_gemm"):
                f = getattr(L, name)
                f.argtypes, f.restype = gemm_args, ctypes.c_int
            L.gmxfp8_quantize.argtypes, L.gmxfp8_quantize.restype = [_P, _P, _P, _I64, _I64, _P], ctypes.c_int
            L.gnf4_grouped_gemm_noalloc.argtypes = [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _P, _P]
            L.gnf4_grouped_gemm_noalloc.restype = ctypes.c_int
            L.geg_lora_workspace_bytes.argtypes = [_I32, _I64, _I64, _I64, _I32, _I32]
            L.geg_lora_workspace_bytes.restype = _SZ
            for name in ("gnf4_grouped_gemm_lora", "gmxfp4_grouped_gemm_lora"):
                f = getattr(L, name)
                f.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _I64, _I64, _I64, _I32, _I32,
                              _P, _SZ, _P, _P]
                f.restype = ctypes.c_int
            for name in ("gnf4_grouped_dgrad_lora", "gmxfp4_grouped_dgrad_lora"):
                f = getattr(L, name)
                f.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _I64, _I64, _I64, _I32,
                              _I32, _P, _SZ, _P, _P]
                f.restype = ctypes.c_int
            L.geg_route_sort.argtypes = [_P, _I64, _I32, _I32, _P, _I64, _P, _P, _P, _P, _P, _SZ, _P]
            L.geg_route_sort.restype = ctypes.c_int
            L.geg_route_workspace_bytes.argtypes = [_I64, _I32, _I32]
            L.geg_route_workspace_bytes.restype = _SZ
            L.geg_route_combine.argtypes = [_P, _P, _P, _I64, _I32, _I64, _P, _P]
            L.geg_route_combine.restype = ctypes.c_int
            block_args = [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I32, _P, _SZ, _P, _P]
            for name in ("gnf4_expert_block", "gmxfp4_expert_block"):
                f = getattr(L, name)
                f.argtypes, f.restype = block_args, ctypes.c_int
            L.gmxfp4_quantize.argtypes = [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]
            L.geg_route_topk.argtypes = [_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _P, _P]
            L.geg_route_topk_grad.argtypes = [_P, _P, _I32, _P, _P, _I64, _I32, _I32, _I32, _P, _P]
            L.geg_route_combine_grad.argtypes = [_P, _P, _P, _P, _P, _I64, _I32, _I64, _P, _P, _P]
            L.geg_moe_layer_workspace_bytes.argtypes = [_I64, _I32, _I64]
            L.geg_moe_layer_workspace_bytes.restype = _SZ
            for name in ("gmxfp4_quantize", "geg_route_topk", "geg_route_topk_grad", "geg_route_combine_grad"):
                getattr(L, name).restype = ctypes.c_int
            for name in ("gnf4_moe_layer", "gmxfp4_moe_layer"):
                f = getattr(L, name)
                f.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I32, _P, _SZ, _P, _P]
                f.restype = ctypes.c_int
            dense = [_P, _P, _P, _P, _I32, _I64, _I64, _I64, _I32, _I32, _P, _SZ, _P, _P]
            for name in ("geg_grouped_gemm", "geg_grouped_dgrad", "geg_grouped_wgrad"):
                f = getattr(L, name)
                f.argtypes, f.restype = dense, ctypes.c_int
            L.geg_grouped_wgrad.argtypes = [_P, _P, _P, _P, _I32, _I32, _I64, _I64, _I64, _I32, _P, _SZ, _P, _P]
            L.geg_request_lora.argtypes = [_P, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I64, _I32, _I32,
                                           _P, _SZ, _P]
            L.geg_request_lora.restype = ctypes.c_int
            L.geg_grouped_workspace_bytes.argtypes = [_I32, _I64, _I64, _I64, _I32]
            L.geg_grouped_workspace_bytes.restype = _SZ
            L.geg_request_lora_workspace_bytes.argtypes = [_I64, _I64, _I32, _I32]
            L.geg_request_lora_workspace_bytes.restype = _SZ
            L.geg_lora_dropout_workspace_bytes.argtypes = [_I32, _I64, _I64, _I64, _I32, _I32]
            L.geg_lora_dropout_workspace_bytes.restype = _SZ
            drop = [ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, _P]
            for fmt in ("gnf4", "gmxfp4"):
                for way, after in (("gemm", 7), ("dgrad", 9)):   # p, seed, offset, rng behind the scale
                    f, plain = getattr(L, f"{fmt}_grouped_{way}_lora_dropout"), getattr(L, f"{fmt}_grouped_{way}_lora").argtypes
                    f.argtypes, f.restype = [*plain[:after], *drop, *plain[after:]], ctypes.c_int
            L.geg_dropout.argtypes = [_P, _P, _P, _I32, _I64, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, _P, _P]
            L.geg_dropout.restype = ctypes.c_int
            L.geg_workspace_bytes.argtypes = [_I32, _I64, _I64, _I64, _I32, _P]
            L.geg_workspace_bytes.restype = _SZ
            L.geg_workspace_init.argtypes, L.geg_workspace_init.restype = [_P, _SZ, _P], ctypes.c_int
            L.geg_read_device_error.argtypes = [_P, ctypes.POINTER(ctypes.c_int32), _P]
            L.geg_read_device_error.restype = ctypes.c_int
            for name in ("gnf4_dequant", "gmxfp4_dequant"):
                f = getattr(L, name)
                f.argtypes, f.restype = [_P, _P, _P, _P, _P, _I64, _I64, _I32, _P], ctypes.c_int
            L.gnf4_quantize.argtypes, L.gnf4_quantize.restype = [_P, _P, _P, _I64, _I64, _P], ctypes.c_int
            L.geg_status_string.argtypes, L.geg_status_string.restype = [ctypes.c_int], ctypes.c_char_p
            L.geg_last_error.argtypes, L.geg_last_error.restype = [], ctypes.c_char_p
            L.geg_version.argtypes, L.geg_version.restype = [], ctypes.c_int32
            L.geg_launch_count.argtypes, L.geg_launch_count.restype = [], ctypes.c_uint64
            _lib = L
    return _lib


class KernelTimer:
    """Four HIP events (tiled-kernel start/end, decode-kernels start/end) that a
    call records around its kernels when passed through `opts()`; `elapsed_ms()`
    returns (tile_ms, decode_ms), None for kernels the call did not launch."""

    def __init__(self, force_path: int = 0, split_k: int = 0):
        self._hip = ctypes.CDLL("libamdhip64.so")
        self._ev = (ctypes.c_void_p * 4)()
        for i in range(4):
            if self._hip.hipEventCreate(ctypes.byref(self._ev, i * ctypes.sizeof(ctypes.c_void_p))) != 0:
                raise GegError("hipEventCreate failed")
        self._opts = Opts(force_path, split_k, ctypes.cast(self._ev, ctypes.c_void_p))

    def opts(self) -> "Opts":
        return self._opts

    def _ms(self, a, b):
        ms = ctypes.c_float(0.0)
        ok = (self._hip.hipEventSynchronize(ctypes.c_void_p(self._ev[b])) == 0 and
              self._hip.hipEventElapsedTime(ctypes.byref(ms), ctypes.c_void_p(self._ev[a]),
                                            ctypes.c_void_p(self._ev[b])) == 0)
        # events the call did not record fail here; leave no error behind for
        # the next launch on this thread
        self._hip.hipGetLastError()
        return ms.value if ok else None

    def elapsed_ms(self):
        return self._ms(0, 1), self._ms(2, 3)

    def __del__(self):
        try:
            for i in range(4):
                self._hip.hipEventDestroy(ctypes.c_void_p(self._ev[i]))
        except Exception:
            pass


def header_functions() -> list:
    """Names of every function declared in include/geg.h."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b((?:geg|gnf4|gmxfp4)_\w+)\s*\(", txt)))


def _check(status: int) -> None:
    if status != 0:
        raise GegError(status, lib().geg_last_error().decode(errors="replace"))


def _check_device_errors(ws, check_errors: bool, stream) -> None:
    """With check_errors, wait for the call, read the workspace's device error word
    and raise GegDeviceError if any bit is set (the word is cleared first, so the
    next call starts clean). Without it, flagged conditions are visible only
    through Workspace.read_error()."""
    if not check_errors:
        return
    bits = ws.read_error(stream)
    if bits:
        ws.reset(stream)
        raise GegDeviceError(bits)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:   # the current one, without building a torch.cuda.Stream, which takes 2.5 us
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _require_gpu(*ts):
    for t in ts:
        if t is not None and t.device.type != "cuda":
            raise GegError(4, "tensors must be on the GPU: this library has no CPU path "
                              "(the CPU oracle under oracle/ is the reference for host data)")


def _check_tensor(t, name, dtype, shape):
    """dtype, shape and dense row-major layout of one operand: the C entry points
    take bare pointers and sizes, so this is the only place they can be checked."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise GegError(2, f"{name}: expected a contiguous {dtype} tensor of shape {list(shape)}, got "
                          f"{t.dtype} {list(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}")


def _check_packed(nf4: bool, w, scales, E, N, K, wname, sname):
    """Packed 4-bit weights [E, N, K/2] with fp32 absmax [E, N, K/64] (NF4) or
    e8m0 bytes [E, N, K/32] (MXFP4)."""
    import torch
    _check_tensor(w, wname, torch.uint8, (E, N, K // 2))
    if nf4:
        _check_tensor(scales, sname, torch.float32, (E, N, K // 64))
    else:
        _check_tensor(scales, sname, torch.uint8, (E, N, K // 32))


def geg_version() -> int:
    return lib().geg_version()


def geg_launch_count() -> int:
    return lib().geg_launch_count()


def geg_workspace_bytes(op, M, N, K, E, opts: Opts | None = None) -> int:
    return lib().geg_workspace_bytes(op, M, N, K, E, ctypes.byref(opts) if opts else None)


class Workspace:
    """A device workspace (torch-allocated uint8 buffer), zeroed once on creation
    and grown on demand. One workspace must not be shared by concurrent calls; calls
    that are ordered may come on any streams. Memory that growing replaces is not
    reused before the streams that it was used on are done with it, and what a
    captured graph uses lives as long as the workspace."""

    def __init__(self, nbytes: int = 1 << 20, device=None):
        import torch
        self._start(device)
        self.ensure(nbytes)
        if not torch.cuda.is_current_stream_capturing():   # zeroed, whichever stream the first call comes on
            torch.cuda.current_stream(self.device).synchronize()

    def _start(self, device):
        import torch
        device = torch.device("cuda" if device is None else device)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        self.buf = None
        self._users = set()      # streams that the buffer was allocated or used on
        self._captured = False   # by a graph
        self._kept = []          # earlier buffers of captured graphs

    def ensure(self, nbytes: int, stream=None):
        """At least nbytes for a call on `stream` (None: the current one)."""
        import torch
        nbytes = max(256, (int(nbytes) + 255) & ~255)
        with _allocating(stream):
            raw = torch._C._cuda_getCurrentRawStream(self.device.index)
            if self.buf is None or self.buf.numel() < nbytes:
                if self._captured:
                    self._kept.append(self.buf)
                self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
                self._users, self._captured = {raw}, False
                _check(lib().geg_workspace_init(_ptr(self.buf), nbytes, ctypes.c_void_p(raw)))
            elif raw not in self._users:
                self._users.add(raw)
                self.buf.record_stream(torch.cuda.current_stream(self.device))
            if not self._captured:
                self._captured = torch.cuda.is_current_stream_capturing()
        return self

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def read_error(self, stream=None) -> int:
        code = ctypes.c_int32(0)
        _check(lib().geg_read_device_error(_ptr(self.buf), ctypes.byref(code), _stream(stream)))
        return code.value

    def reset(self, stream=None):
        _check(lib().geg_workspace_init(_ptr(self.buf), self.nbytes, _stream(stream)))


class _OwnWorkspace(Workspace):
    """One of this library's own, for one thread and stream: no memory before the first
    ensure(), on that stream."""

    def __init__(self, device):
        self._start(device)

    def take(self, nbytes):
        """Memory of one captured call, whose error word nobody can read: not zeroed."""
        import torch
        self.buf = torch.empty(max(256, nbytes), dtype=torch.uint8, device=self.device)
        return self


class _PerThread(threading.local):
    def __init__(self):
        self.of = {}


_own_ws = _PerThread()


def _workspace(ws, need, device, stream, check_errors=False):
    """The caller's workspace, or one of this library's own for the host thread, device and
    stream: calls on two streams never share one, nor calls of two threads, whose launches on
    one stream may come in turns (a call may be several). A call on a stream that is being
    captured gets one from the graph's memory pool, as that stream's allocation: what takes
    the memory next in the graph runs on the same stream, behind the call. With check_errors
    the error word of an own one is cleared first: earlier calls may have left it set."""
    import torch
    with _allocating(stream):   # the call's stream is the current one in here
        if ws is not None:
            return ws.ensure(need)
        if torch.cuda.is_current_stream_capturing():
            return _OwnWorkspace(device).take(need)
        key = (device.index, torch._C._cuda_getCurrentRawStream(device.index))
        ws = _own_ws.of.get(key)
        if ws is None:
            ws = _own_ws.of[key] = _OwnWorkspace(device)
        if ws.buf is None or ws.buf.numel() < need:
            ws.ensure(max(need, 1 << 20))
        if check_errors:
            ws.reset()
    return ws


def _gemm(fn_name, op, a, sizes, wq, scales, out, workspace, opts, stream, check_errors=False):
    import torch
    M, K = a.shape
    E, N = wq.shape[0], wq.shape[1]
    _check_tensor(a, "a", torch.bfloat16, (M, K))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_packed(op == GEG_OP_NF4_FWD, wq, scales, E, N, K, "weights", "scales")
    _check_tensor(out, "out", torch.bfloat16, (M, N))
    _require_gpu(a, sizes, wq, scales, out)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    need = geg_workspace_bytes(op, M, N, K, E, opts)
    ws = _workspace(workspace, need, a.device, stream, check_errors)
    f = getattr(lib(), fn_name)
    _check(f(_ptr(a), _ptr(sizes), _ptr(wq), _ptr(scales), _ptr(out), M, N, K, E,
             _ptr(ws.buf), ws.nbytes, ctypes.byref(opts) if opts else None, _stream(stream)))
    _check_device_errors(ws, check_errors, stream)
    return out


def gnf4_grouped_gemm(a, sizes, w, absmax, out=None, workspace: Workspace | None = None,
                      opts: Opts | None = None, stream=None, check_errors: bool = False):
    """a bf16 [M,K] (rows grouped by expert), sizes int32 [E], w uint8 [E,N,K/2],
    absmax fp32 [E,N,K/64] -> out bf16 [M,N].

    Conditions the kernels flag on the device (negative sizes, sum(sizes) > M,
    fp16 overflow on a decode path) are clamped there and recorded in the
    workspace's error word; check_errors=True waits for the call and raises
    GegDeviceError when the word is set (the same holds for every wrapper below)."""
    return _gemm("gnf4_grouped_gemm", GEG_OP_NF4_FWD, a, sizes, w, absmax, out, workspace, opts, stream,
                 check_errors)


def gnf4_grouped_gemm_noalloc(a, sizes, w, absmax, out, error_word=None, opts: Opts | None = None, stream=None):
    """gnf4_grouped_gemm without a workspace, for callers that cannot allocate device
    memory: the library's kernels take their scratch from a library-held static
    array (144 MiB per GPU; larger calls raise GEG_ERR_WORKSPACE), so `out` must be
    given. error_word: None or a device int32 tensor of one element that receives
    the call's device error bits (OR-ed in). Calls that overlap on one GPU race on
    the shared array; calls ordered on one stream do not."""
    import torch
    M, K = a.shape
    E, N = w.shape[0], w.shape[1]
    _check_tensor(a, "a", torch.bfloat16, (M, K))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_packed(True, w, absmax, E, N, K, "weights", "absmax")
    _check_tensor(out, "out", torch.bfloat16, (M, N))
    _check_tensor(error_word, "error_word", torch.int32, (1,))
    _require_gpu(a, sizes, w, absmax, out, error_word)
    _check(lib().gnf4_grouped_gemm_noalloc(_ptr(a), _ptr(sizes), _ptr(w), _ptr(absmax), _ptr(out), M, N, K, E,
                                           _ptr(error_word), ctypes.byref(opts) if opts else None, _stream(stream)))
    return out


def gmxfp4_grouped_gemm(a, sizes, blocks, scales, out=None, workspace: Workspace | None = None,
                        opts: Opts | None = None, stream=None, check_errors: bool = False):
    """a bf16 [M,K], sizes int32 [E], blocks uint8 [E,N,K/2] (or [E,N,K/32,16]),
    scales uint8 [E,N,K/32] -> out bf16 [M,N]."""
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    return _gemm("gmxfp4_grouped_gemm", GEG_OP_MXFP4_FWD, a, sizes, blocks, scales, out, workspace,
                 opts, stream, check_errors)


def _dgrad(fn_name, op, dy, sizes, w, scales, dx, workspace, opts, stream, check_errors=False):
    import torch
    M, N = dy.shape
    E, K = w.shape[0], w.shape[2] * 2
    _check_tensor(dy, "dy", torch.bfloat16, (M, N))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_packed(op == GEG_OP_NF4_DGRAD, w, scales, E, N, K, "weights", "scales")
    _check_tensor(dx, "dx", torch.bfloat16, (M, K))
    _require_gpu(dy, sizes, w, scales, dx)
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
    need = geg_workspace_bytes(op, M, N, K, E, opts)
    ws = _workspace(workspace, need, dy.device, stream, check_errors)
    _check(getattr(lib(), fn_name)(_ptr(dy), _ptr(sizes), _ptr(w), _ptr(scales), _ptr(dx), M, N, K, E,
                                   _ptr(ws.buf), ws.nbytes, ctypes.byref(opts) if opts else None,
                                   _stream(stream)))
    _check_device_errors(ws, check_errors, stream)
    return dx


def gnf4_grouped_dgrad(dy, sizes, w, absmax, dx=None, workspace: Workspace | None = None,
                       opts: Opts | None = None, stream=None, check_errors: bool = False):
    """dy bf16 [M,N], w uint8 [E,N,K/2], absmax fp32 [E,N,K/64] -> dx bf16 [M,K]."""
    return _dgrad("gnf4_grouped_dgrad", GEG_OP_NF4_DGRAD, dy, sizes, w, absmax, dx, workspace, opts, stream,
                  check_errors)


def gmxfp4_grouped_dgrad(dy, sizes, blocks, scales, dx=None, workspace: Workspace | None = None,
                         opts: Opts | None = None, stream=None, check_errors: bool = False):
    """dy bf16 [M,N], blocks uint8 [E,N,K/2], scales uint8 [E,N,K/32] -> dx bf16 [M,K]."""
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    return _dgrad("gmxfp4_grouped_dgrad", GEG_OP_MXFP4_DGRAD, dy, sizes, blocks, scales, dx, workspace, opts,
                  stream, check_errors)


def gmxfp4_w4a8_grouped_gemm(a, sizes, blocks, scales, out=None, workspace: Workspace | None = None,
                             opts: Opts | None = None, stream=None, check_errors: bool = False):
    """W4A8: a bf16 [M,K] quantised on the device to MXFP8 (e4m3, one e8m0 scale per
    32 k) times MXFP4 blocks uint8 [E,N,K/2] (or [E,N,K/32,16]) with scales uint8
    [E,N,K/32] on the block-scaled matrix instruction -> out bf16 [M,N]."""
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    return _gemm("gmxfp4_w4a8_grouped_gemm", GEG_OP_MXFP4_W4A8, a, sizes, blocks, scales, out, workspace,
                 opts, stream, check_errors)


def gmxfp8_quantize(a, stream=None):
    """a bf16 [M,K] (K % 32 == 0) -> (e4m3 codes uint8 [M,K], e8m0 scales uint8 [M,K/32])."""
    import torch
    M, K = a.shape
    _check_tensor(a, "a", torch.bfloat16, (M, K))
    _require_gpu(a)
    codes = torch.empty((M, K), dtype=torch.uint8, device=a.device)
    scales = torch.empty((M, K // 32), dtype=torch.uint8, device=a.device)
    _check(lib().gmxfp8_quantize(_ptr(a), _ptr(codes), _ptr(scales), M, K, _stream(stream)))
    return codes, scales


def _check_lora(x, sizes, lora_a, lora_b):
    import torch
    M, K = x.shape
    E, r = lora_a.shape[0], lora_a.shape[1]
    N = lora_b.shape[1]
    _check_tensor(x, "x", torch.bfloat16, (M, K))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_tensor(lora_a, "lora_a", torch.float32, (E, r, K))
    _check_tensor(lora_b, "lora_b", torch.float32, (E, N, r))
    return M, N, K, E, r


def _lora_call(name, dropout, x):
    """The entry point of an adapter call and what dropout = (p, seed, offset) of x adds to its arguments."""
    if dropout is None:
        return getattr(lib(), name), lib().geg_lora_workspace_bytes, ()
    p, seed, offset = dropout
    seed, offset, rng = _seed(seed, offset)
    if rng is not None:
        _on_device(x, rng)
    return (getattr(lib(), name + "_dropout"), lib().geg_lora_dropout_workspace_bytes, (float(p), seed, offset, _ptr(rng)))


def _gemm_lora(fmt, a, sizes, w, scales, lora_a, lora_b, scale, out, u, workspace, opts, stream,
               check_errors=False, dropout=None):
    import torch
    M, N, K, E, r = _check_lora(a, sizes, lora_a, lora_b)
    _check_packed(fmt == "nf4", w, scales, E, N, K, "weights", "scales")
    fn, need, drop = _lora_call("gnf4_grouped_gemm_lora" if fmt == "nf4" else "gmxfp4_grouped_gemm_lora", dropout, a)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    if u is None:
        u = torch.empty((M, r), dtype=torch.float32, device=a.device)
    _check_tensor(out, "out", torch.bfloat16, (M, N))
    _check_tensor(u, "u", torch.float32, (M, r))
    _require_gpu(a, sizes, w, scales, lora_a, lora_b, out, u)
    op = GEG_OP_NF4_FWD if fmt == "nf4" else GEG_OP_MXFP4_FWD
    ws = _workspace(workspace, need(op, M, N, K, E, r), a.device, stream, check_errors)
    _check(fn(_ptr(a), _ptr(sizes), _ptr(w), _ptr(scales), _ptr(lora_a), _ptr(lora_b), float(scale), *drop, _ptr(out),
              _ptr(u), M, N, K, E, r, _ptr(ws.buf), ws.nbytes, ctypes.byref(opts) if opts else None, _stream(stream)))
    _check_device_errors(ws, check_errors, stream)
    return out, u


def gnf4_grouped_gemm_lora(a, sizes, w, absmax, lora_a, lora_b, scale: float, out=None, u=None,
                           workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                           check_errors: bool = False):
    """out = a_e W_e^T + scale (a_e A_e^T) B_e^T per expert, the adapter delta added
    to the fp32 accumulators before the bf16 rounding; lora_a fp32 [E, r, K],
    lora_b fp32 [E, N, r]. Returns (out bf16 [M, N], u = a A_e^T fp32 [M, r])."""
    return _gemm_lora("nf4", a, sizes, w, absmax, lora_a, lora_b, scale, out, u, workspace, opts, stream,
                      check_errors)


def gmxfp4_grouped_gemm_lora(a, sizes, blocks, scales, lora_a, lora_b, scale: float, out=None, u=None,
                             workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                             check_errors: bool = False):
    """The same on MXFP4 weights (blocks uint8 [E, N, K/2], scales uint8 [E, N, K/32])."""
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    return _gemm_lora("mxfp4", a, sizes, blocks, scales, lora_a, lora_b, scale, out, u, workspace, opts, stream,
                      check_errors)


def _dgrad_lora(fmt, dy, sizes, w, scales, x, lora_a, lora_b, u, scale, dx, grad_a, grad_b, workspace, opts,
                stream, check_errors=False, dropout=None):
    import torch
    M, N, K, E, r = _check_lora(x, sizes, lora_a, lora_b)
    _check_packed(fmt == "nf4", w, scales, E, N, K, "weights", "scales")
    _check_tensor(dy, "dy", torch.bfloat16, (M, N))
    _check_tensor(u, "u", torch.float32, (M, r))
    fn, need, drop = _lora_call("gnf4_grouped_dgrad_lora" if fmt == "nf4" else "gmxfp4_grouped_dgrad_lora", dropout, x)
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
    if grad_a is None:
        grad_a = torch.empty((E, r, K), dtype=torch.float32, device=dy.device)
    if grad_b is None:
        grad_b = torch.empty((E, N, r), dtype=torch.float32, device=dy.device)
    _check_tensor(dx, "dx", torch.bfloat16, (M, K))
    _check_tensor(grad_a, "grad_a", torch.float32, (E, r, K))
    _check_tensor(grad_b, "grad_b", torch.float32, (E, N, r))
    _require_gpu(dy, sizes, w, scales, x, lora_a, lora_b, u, dx, grad_a, grad_b)
    op = GEG_OP_NF4_DGRAD if fmt == "nf4" else GEG_OP_MXFP4_DGRAD
    ws = _workspace(workspace, need(op, M, N, K, E, r), dy.device, stream, check_errors)
    _check(fn(_ptr(dy), _ptr(sizes), _ptr(w), _ptr(scales), _ptr(x), _ptr(lora_a), _ptr(lora_b), _ptr(u),
              float(scale), *drop, _ptr(dx), _ptr(grad_a), _ptr(grad_b), M, N, K, E, r, _ptr(ws.buf), ws.nbytes,
              ctypes.byref(opts) if opts else None, _stream(stream)))
    _check_device_errors(ws, check_errors, stream)
    return dx, grad_a, grad_b


def gnf4_grouped_dgrad_lora(dy, sizes, w, absmax, x, lora_a, lora_b, u, scale: float, dx=None, grad_a=None,
                            grad_b=None, workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                            check_errors: bool = False):
    """Backward of gnf4_grouped_gemm_lora: (dx = dy W_e + scale (dy B_e) A_e bf16
    [M, K], grad_a fp32 [E, r, K], grad_b fp32 [E, N, r])."""
    return _dgrad_lora("nf4", dy, sizes, w, absmax, x, lora_a, lora_b, u, scale, dx, grad_a, grad_b, workspace,
                       opts, stream, check_errors)


def gmxfp4_grouped_dgrad_lora(dy, sizes, blocks, scales, x, lora_a, lora_b, u, scale: float, dx=None, grad_a=None,
                              grad_b=None, workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                              check_errors: bool = False):
    """The same on MXFP4 weights."""
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    return _dgrad_lora("mxfp4", dy, sizes, blocks, scales, x, lora_a, lora_b, u, scale, dx, grad_a, grad_b,
                       workspace, opts, stream, check_errors)


def grouped_linear_lora(a, sizes, w, scales, lora_a, lora_b, scale: float, fmt: str = "nf4",
                        check_errors: bool = False, dropout: float = 0.0, seed=None, offset: int = 0):
    """The grouped 4-bit projection with a trainable low-rank delta at the
    pre-activation point, as a torch autograd op: out = a_e W_e^T + scale *
    (a_e A_e^T) B_e^T per expert. Backward: dA (through the dgrad kernel and the
    adapter kernels), d lora_a, d lora_b (fp32); the 4-bit weights are frozen.
    check_errors=True makes both directions raise GegDeviceError on a flagged
    device condition (see gnf4_grouped_gemm). dropout > 0 drops values of the adapter's
    input (the projection's stays whole) by philox_dropout's mask for seed and offset over
    a, which both directions draw anew; seed as in dropout()."""
    if dropout:
        if seed is None:
            raise GegError(8, "dropout needs a seed: an int, or a device int64 tensor {seed, offset}")
        import torch
        rng = seed if isinstance(seed, torch.Tensor) else None
        return _GroupedLinearLora.apply(a, sizes, w, scales, lora_a, lora_b, float(scale), fmt, bool(check_errors),
                                        (float(dropout), None if rng is not None else seed, int(offset)), rng)
    return _GroupedLinearLora.apply(a, sizes, w, scales, lora_a, lora_b, float(scale), fmt, bool(check_errors), None, None)


def grouped_linear(a, sizes, w, scales, fmt: str = "nf4", check_errors: bool = False):
    """The grouped 4-bit GEMM as a differentiable op (torch autograd): out = per
    expert a_e W_e^T; the backward returns dA = per expert dOut_e W_e through the
    library's dgrad kernel on the same packed bytes. The 4-bit weights are frozen
    (no gradient), as in 4-bit adapter training. check_errors=True makes both
    directions raise GegDeviceError on a flagged device condition."""
    return _GroupedLinear.apply(a, sizes, w, scales, fmt, bool(check_errors))


def _make_grouped_linear():
    import torch

    class GroupedLinear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, sizes, w, scales, fmt, check_errors):
            ctx.save_for_backward(sizes, w, scales)
            ctx.fmt, ctx.check_errors = fmt, check_errors
            fn = gnf4_grouped_gemm if fmt == "nf4" else gmxfp4_grouped_gemm
            return fn(a, sizes, w, scales, check_errors=check_errors)

        @staticmethod
        def backward(ctx, grad_out):
            sizes, w, scales = ctx.saved_tensors
            fn = gnf4_grouped_dgrad if ctx.fmt == "nf4" else gmxfp4_grouped_dgrad
            da = (fn(grad_out.contiguous().to(torch.bfloat16), sizes, w, scales, check_errors=ctx.check_errors)
                  if ctx.needs_input_grad[0] else None)
            return da, None, None, None, None, None

    return GroupedLinear


def _make_grouped_linear_lora():
    import torch

    class GroupedLinearLora(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, sizes, w, scales, lora_a, lora_b, scale, fmt, check_errors, dropout, rng):
            if dropout is not None and rng is not None:
                dropout = (dropout[0], rng, dropout[2])
            out, u = _gemm_lora(fmt, a, sizes, w, scales, lora_a, lora_b, scale, None, None, None, None, None,
                                check_errors, dropout)
            ctx.save_for_backward(a, sizes, w, scales, lora_a, lora_b, u, *(() if rng is None else (rng,)))
            ctx.fmt, ctx.scale, ctx.check_errors = fmt, scale, check_errors
            ctx.dropout = None if dropout is None else (dropout[0], None if rng is not None else dropout[1], dropout[2])
            return out

        @staticmethod
        def backward(ctx, grad_out):
            a, sizes, w, scales, lora_a, lora_b, u, *rng = ctx.saved_tensors
            dropout = ctx.dropout
            if rng:
                dropout = (dropout[0], rng[0], dropout[2])
            da, ga, gb = _dgrad_lora(ctx.fmt, grad_out.contiguous(), sizes, w, scales, a, lora_a, lora_b, u, ctx.scale,
                                     None, None, None, None, None, None, ctx.check_errors, dropout)
            return ((da if ctx.needs_input_grad[0] else None), None, None, None, ga, gb, None, None, None, None, None)

    return GroupedLinearLora


class _LazyFn:
    def __init__(self, make):
        self._make = make
        self._f = None

    def apply(self, *args):
        if self._f is None:
            self._f = self._make()
        return self._f.apply(*args)


_GroupedLinear = _LazyFn(_make_grouped_linear)
_GroupedLinearLora = _LazyFn(_make_grouped_linear_lora)


def _block(fn_name, op, a, sizes, w13, s13, w2, s2, out, workspace, opts, stream, check_errors=False):
    import torch
    M, H = a.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    nf4 = op == GEG_OP_NF4_BLOCK
    _check_tensor(a, "a", torch.bfloat16, (M, H))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_packed(nf4, w13, s13, E, 2 * I, H, "w13", "scales13")
    _check_packed(nf4, w2, s2, E, H, I, "w2", "scales2")
    _check_tensor(out, "out", torch.bfloat16, (M, H))
    _require_gpu(a, sizes, w13, s13, w2, s2, out)
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=a.device)
    need = geg_workspace_bytes(op, M, H, I, E, opts)
    ws = _workspace(workspace, need, a.device, stream, check_errors)
    _check(getattr(lib(), fn_name)(_ptr(a), _ptr(sizes), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
                                   _ptr(out), M, H, I, E, _ptr(ws.buf), ws.nbytes,
                                   ctypes.byref(opts) if opts else None, _stream(stream)))
    _check_device_errors(ws, check_errors, stream)
    return out


def gnf4_expert_block(a, sizes, w13, absmax13, w2, absmax2, out=None,
                      workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                      check_errors: bool = False):
    """Fused SwiGLU expert MLP: a bf16 [M,H], w13 uint8 [E,2I,H/2] (rows 2i gate,
    2i+1 up), absmax13 fp32 [E,2I,H/64], w2 uint8 [E,H,I/2], absmax2 fp32
    [E,H,I/64] -> out bf16 [M,H]."""
    return _block("gnf4_expert_block", GEG_OP_NF4_BLOCK, a, sizes, w13, absmax13, w2, absmax2, out,
                  workspace, opts, stream, check_errors)


def gmxfp4_expert_block(a, sizes, blocks13, scales13, blocks2, scales2, out=None,
                        workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                        check_errors: bool = False):
    """The same block on MXFP4: blocks13 uint8 [E,2I,H/2], scales13 uint8
    [E,2I,H/32], blocks2 uint8 [E,H,I/2], scales2 uint8 [E,H,I/32]."""
    if blocks13.dim() == 4:
        blocks13 = blocks13.reshape(blocks13.shape[0], blocks13.shape[1], -1)
    if blocks2.dim() == 4:
        blocks2 = blocks2.reshape(blocks2.shape[0], blocks2.shape[1], -1)
    return _block("gmxfp4_expert_block", GEG_OP_MXFP4_BLOCK, a, sizes, blocks13, scales13, blocks2,
                  scales2, out, workspace, opts, stream, check_errors)


def route_sort(topk_ids, E: int, x=None, workspace: Workspace | None = None, stream=None,
               check_errors: bool = False):
    """Device-side routing sort of topk_ids int32 [T, k] over E experts.

    Returns (sizes int32 [E], row_of int32 [T*k], src_of int32 [T*k], x_sorted):
    entries ordered by expert, then by t*k + slot; x_sorted bf16 [T*k, H] holds
    x[src_of[r] // k] in sorted row r when x (bf16 [T, H]) is given, else None."""
    import torch
    T, k = topk_ids.shape
    _check_tensor(topk_ids, "topk_ids", torch.int32, (T, k))
    if x is not None:
        _check_tensor(x, "x", torch.bfloat16, (T, x.shape[1]))
    _on_device(topk_ids, x)
    dev = topk_ids.device
    xs = None
    H = 0
    with _allocating(stream):
        sizes = torch.empty((E,), dtype=torch.int32, device=dev)
        row_of = torch.empty((T * k,), dtype=torch.int32, device=dev)
        src_of = torch.empty((T * k,), dtype=torch.int32, device=dev)
        if x is not None:
            H = x.shape[1]
            xs = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev)
        ws = _workspace(workspace, lib().geg_route_workspace_bytes(T, k, E), dev, None, check_errors)
    raw = _raw_stream(stream, topk_ids)
    _check(lib().geg_route_sort(_ptr(topk_ids), T, k, E, _ptr(x), H, _ptr(sizes), _ptr(row_of),
                                _ptr(src_of), _ptr(xs), _ptr(ws.buf), ws.nbytes, raw))
    _outlive(stream, sizes, row_of, src_of, xs)
    _check_device_errors(ws, check_errors, stream)
    return sizes, row_of, src_of, xs


def route_combine(y, row_of, weights, k: int, out=None, stream=None):
    """out bf16 [T, N] = sum over slots of weights[t, s] * y[row_of[t*k + s]] (fp32 in
    slot order); y bf16 [T*k, N] in routing-sort order, weights fp32 [T, k] or None."""
    import torch
    T = row_of.numel() // k
    N = y.shape[1]
    _check_tensor(row_of, "row_of", torch.int32, (T * k,))
    _check_tensor(y, "y", torch.bfloat16, (T * k, N))
    _check_tensor(weights, "weights", torch.float32, (T, k))
    _check_tensor(out, "out", torch.bfloat16, (T, N))
    _require_gpu(y, row_of, weights, out)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=y.device)
    _check(lib().geg_route_combine(_ptr(y), _ptr(row_of), _ptr(weights), T, k, N, _ptr(out), _stream(stream)))
    return out


def _dequant(fn_name, wq, scales, bf16, f16, stream):
    import torch
    E, N, K = wq.shape[0], wq.shape[1], wq.shape[2] * 2
    _check_packed(fn_name == "gnf4_dequant", wq, scales, E, N, K, "weights", "scales")
    _require_gpu(wq, scales)
    f32 = torch.empty((E, N, K), dtype=torch.float32, device=wq.device)
    ob = torch.empty((E, N, K), dtype=torch.bfloat16, device=wq.device) if bf16 else None
    oh = torch.empty((E, N, K), dtype=torch.float16, device=wq.device) if f16 else None
    _check(getattr(lib(), fn_name)(_ptr(wq), _ptr(scales), _ptr(f32), _ptr(ob), _ptr(oh), N, K, E,
                                   _stream(stream)))
    return f32, ob, oh


def gnf4_dequant(w, absmax, bf16=True, f16=True, stream=None):
    """Decode NF4 [E,N,K/2] + [E,N,K/64] to (fp32, bf16|None, fp16|None) [E,N,K]."""
    return _dequant("gnf4_dequant", w, absmax, bf16, f16, stream)


def gmxfp4_dequant(blocks, scales, bf16=True, f16=True, stream=None):
    """Decode MXFP4 [E,N,K/2] + [E,N,K/32] to (fp32, bf16|None, fp16|None) [E,N,K]."""
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    return _dequant("gmxfp4_dequant", blocks, scales, bf16, f16, stream)


def gnf4_quantize(w, stream=None):
    """NF4-pack fp32 weights [..., K] on the GPU -> (codes uint8 [..., K/2], absmax fp32 [..., K/64])."""
    import torch
    _require_gpu(w)
    if w.dtype != torch.float32 or not w.is_contiguous():
        raise GegError(2, "gnf4_quantize expects a contiguous fp32 tensor")
    K = w.shape[-1]
    rows = w.numel() // K
    codes = torch.empty(w.shape[:-1] + (K // 2,), dtype=torch.uint8, device=w.device)
    absmax = torch.empty(w.shape[:-1] + (K // 64,), dtype=torch.float32, device=w.device)
    _check(lib().gnf4_quantize(_ptr(w), _ptr(codes), _ptr(absmax), rows, K, _stream(stream)))
    return codes, absmax


# ----------------------------------------------------------------------------- MXFP4 packer, gate, few-token layer
_DTYPES = {}


def _dtype(t, name):
    """GEG_BF16 / GEG_F16 / GEG_F32 of a tensor, refused otherwise."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise GegError(2, f"{name}: expected a bfloat16, float16 or float32 tensor, got {t.dtype}")
    return code


def _on_device(ref, *ts):
    """Every tensor on ref's device, and that the current one: kernels launch on the
    current device's streams."""
    import torch
    dev = ref.get_device()   # -1 unless on a GPU
    if dev < 0:
        _require_gpu(ref)
    for t in ts:
        if t is not None and t.get_device() != dev:
            _require_gpu(t)
            raise GegError(4, f"tensors on several devices: {ref.device} and {t.device}")
    if dev != torch._C._cuda_getDevice():
        raise GegError(4, f"tensors are on {ref.device} but the current device is "
                          f"cuda:{torch.cuda.current_device()}: call under torch.cuda.device(...)")


def _raw_stream(stream, ref):
    """The hipStream_t of a call: the given stream's, or the current one of ref's device
    (read without building a torch.cuda.Stream, which costs as much as a launch)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(ref.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _addr(t):
    return None if t is None else t.data_ptr()


_NO_CHANGE = contextlib.nullcontext()


class _OnStream:
    """torch.cuda.stream(stream) without its checks, which cost as much as a call."""
    __slots__ = ("stream", "before")

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        from torch import _C
        s = self.stream
        self.before = _C._cuda_getCurrentStream(_C._cuda_getDevice())
        _C._cuda_setStream(stream_id=s.stream_id, device_index=s.device_index, device_type=s.device_type)

    def __exit__(self, *_):
        from torch import _C
        at, index, kind = self.before
        _C._cuda_setStream(stream_id=at, device_index=index, device_type=kind)


def _allocating(stream):
    """Context in which a call on `stream` allocates: memory for another stream than the
    current one comes from that stream's pool, where only its own earlier work (or work
    that was recorded on it) may still use it."""
    if stream is None:
        return _NO_CHANGE
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    return _OnStream(stream)


def _outlive(stream, *ts):
    """Results that a call on another stream allocated there stay allocated until the
    current stream, where they are going to be used, is done with them."""
    if stream is None:
        return
    import torch
    here = torch.cuda.current_stream()
    for t in ts:
        if t is not None:
            t.record_stream(here)


def gmxfp4_quantize(x, values: bool = False, stream=None):
    """MXFP4-pack x [..., K] (bf16, fp16 or fp32; K % 32 == 0) on the GPU -> (blocks uint8
    [..., K/2], scales uint8 [..., K/32]), with values=True also the values that the
    codes stand for, in x's type (exact): what a quantisation-aware forward pass uses.

    A 2-D x may have rows further apart than K (a slice of columns); its rows have to
    start at multiples of 16 bytes. Blocks holding an inf or NaN decode to NaN."""
    import torch
    dt = _dtype(x, "x")
    K = x.shape[-1] if x.dim() else 0
    if K <= 0 or K % 32:
        raise GegError(2, f"x: the last dimension must be a positive multiple of 32, got shape {list(x.shape)}")
    rows = x.numel() // K
    if x.is_contiguous():
        ld = K
    elif x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= K:
        ld = x.stride(0)
    else:
        raise GegError(2, f"x: expected a contiguous tensor, or a 2-D one of contiguous rows, got strides "
                          f"{list(x.stride())} of shape {list(x.shape)}")
    _on_device(x)
    lead = x.shape[:-1]
    with _allocating(stream):
        codes = x.new_empty(lead + (K // 2,), dtype=torch.uint8)
        scales = codes.new_empty(lead + (K // 32,))
        vals = x.new_empty(x.shape) if values else None
    _check(lib().gmxfp4_quantize(x.data_ptr(), dt, rows, K, ld, codes.data_ptr(), scales.data_ptr(), _addr(vals),
                                 _raw_stream(stream, x)))
    _outlive(stream, codes, scales, vals)
    return (codes, scales, vals) if values else (codes, scales)


def gmxfp4_w4a4_grouped_gemm(a, sizes, blocks, scales, out=None, workspace: Workspace | None = None,
                             opts: Opts | None = None, stream=None, check_errors: bool = False):
    """W4A4: a bf16 [M, K] quantised to MXFP4 inside the call, times MXFP4 blocks uint8
    [E, N, K/2] (or [E, N, K/32, 16]) with scales uint8 [E, N, K/32], on the block-scaled
    matrix instruction with two 4-bit operands -> out bf16 [M, N]. Rows with an inf or
    NaN come out NaN and flag DEVERR_NON_FINITE."""
    import torch
    if blocks.dim() == 4:
        blocks = blocks.reshape(blocks.shape[0], blocks.shape[1], -1)
    if a.dim() != 2 or blocks.dim() != 3:
        raise GegError(2, "a: expected [M, K], blocks [E, N, K/2]")
    M, K = a.shape
    E, N = blocks.shape[0], blocks.shape[1]
    _check_tensor(a, "a", torch.bfloat16, (M, K))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_packed(False, blocks, scales, E, N, K, "blocks", "scales")
    _check_tensor(out, "out", torch.bfloat16, (M, N))
    _on_device(a, sizes, blocks, scales, out)
    mine = out is None
    L, o = lib(), ctypes.byref(opts) if opts else None
    raw = _raw_stream(stream, a)
    with _allocating(stream):
        if mine:
            out = a.new_empty((M, N))
        ws = _workspace(workspace, L.geg_workspace_bytes(GEG_OP_MXFP4_W4A4, M, N, K, E, o), a.device, None, check_errors)
    _check(L.gmxfp4_w4a4_grouped_gemm(a.data_ptr(), sizes.data_ptr(), blocks.data_ptr(), scales.data_ptr(),
                                      out.data_ptr(), M, N, K, E, ws.buf.data_ptr(), ws.buf.numel(), o, raw))
    if mine:
        _outlive(stream, out)
    _check_device_errors(ws, check_errors, stream)
    return out


def route_topk(logits, k: int, renormalize: bool = True, error_word=None, stream=None):
    """The router's gate: logits [T, E] (bf16, fp16 or fp32) -> (weights fp32 [T, k], ids
    int32 [T, k]): the k largest logits, largest first, ties to the lower expert, and
    their softmax weights, over all experts or renormalised over the chosen ones. NaN
    logits count as -inf and flag DEVERR_NON_FINITE in error_word (None, or a device
    int32 tensor of one element, OR-ed in)."""
    import torch
    dt = _dtype(logits, "logits")
    if logits.dim() != 2 or not logits.is_contiguous():
        raise GegError(2, f"logits: expected a contiguous [T, E] tensor, got {list(logits.shape)}")
    T, E = logits.shape
    _check_tensor(error_word, "error_word", torch.int32, (1,))
    _on_device(logits, error_word)
    with _allocating(stream):
        weights = logits.new_empty((T, k), dtype=torch.float32)
        ids = logits.new_empty((T, k), dtype=torch.int32)
    _check(lib().geg_route_topk(logits.data_ptr(), dt, T, E, k, int(renormalize), weights.data_ptr(), ids.data_ptr(),
                                _addr(error_word), _raw_stream(stream, logits)))
    _outlive(stream, weights, ids)
    return weights, ids


def route_topk_grad(dweights, logits, ids, weights, renormalize: bool = True, stream=None):
    """Gradient of route_topk's weights: dweights fp32 [T, k] and the forward's logits,
    ids and weights -> dlogits [T, E] in the logits' type."""
    import torch
    dt = _dtype(logits, "logits")
    if logits.dim() != 2 or not logits.is_contiguous() or ids.dim() != 2:
        raise GegError(2, "logits: expected a contiguous [T, E] tensor and ids [T, k]")
    T, E = logits.shape
    k = ids.shape[1]
    _check_tensor(ids, "ids", torch.int32, (T, k))
    _check_tensor(weights, "weights", torch.float32, (T, k))
    _check_tensor(dweights, "dweights", torch.float32, (T, k))
    _on_device(logits, ids, weights, dweights)
    with _allocating(stream):
        dlogits = logits.new_empty((T, E))
    _check(lib().geg_route_topk_grad(dweights.data_ptr(), logits.data_ptr(), dt, ids.data_ptr(), weights.data_ptr(), T,
                                     E, k, int(renormalize), dlogits.data_ptr(), _raw_stream(stream, logits)))
    _outlive(stream, dlogits)
    return dlogits


def route_combine_grad(dout, y, row_of, weights, src_of=None, stream=None):
    """Gradient of route_combine: dout bf16 [T, N], the forward's y bf16 [T*k, N], row_of
    int32 [T*k] and weights fp32 [T, k] -> (dy bf16 [T*k, N], dweights fp32 [T, k]).
    Rows of dy that no entry lands on are set to 0 when route_sort's src_of is given,
    else left as they were allocated."""
    import torch
    if weights.dim() != 2 or dout.dim() != 2:
        raise GegError(2, "weights: expected [T, k], dout [T, N]")
    T, k = weights.shape
    N = dout.shape[1]
    _check_tensor(dout, "dout", torch.bfloat16, (T, N))
    _check_tensor(y, "y", torch.bfloat16, (T * k, N))
    _check_tensor(row_of, "row_of", torch.int32, (T * k,))
    _check_tensor(src_of, "src_of", torch.int32, (T * k,))
    _check_tensor(weights, "weights", torch.float32, (T, k))
    _on_device(dout, y, row_of, weights, src_of)
    with _allocating(stream):
        dy = y.new_empty((T * k, N))
        dw = weights.new_empty((T, k))
    _check(lib().geg_route_combine_grad(dout.data_ptr(), y.data_ptr(), row_of.data_ptr(), _addr(src_of),
                                        weights.data_ptr(), T, k, N, dy.data_ptr(), dw.data_ptr(),
                                        _raw_stream(stream, dout)))
    _outlive(stream, dy, dw)
    return dy, dw


def _moe_layer(nf4, x, topk_ids, topk_weights, w13, s13, w2, s2, out, workspace, opts, stream, check_errors):
    import torch
    if x.dim() != 2 or topk_ids.dim() != 2 or w13.dim() != 3:
        raise GegError(2, "x: expected [T, H], topk_ids [T, k], w13 [E, 2I, H/2]")
    T, H = x.shape
    k = topk_ids.shape[1]
    E, I = w13.shape[0], w13.shape[1] // 2
    _check_tensor(x, "x", torch.bfloat16, (T, H))
    _check_tensor(topk_ids, "topk_ids", torch.int32, (T, k))
    _check_tensor(topk_weights, "topk_weights", torch.float32, (T, k))
    _check_packed(nf4, w13, s13, E, 2 * I, H, "w13", "scales13")
    _check_packed(nf4, w2, s2, E, H, I, "w2", "scales2")
    _check_tensor(out, "out", torch.bfloat16, (T, H))
    _on_device(x, topk_ids, topk_weights, w13, s13, w2, s2, out)
    mine = out is None
    L = lib()
    raw = _raw_stream(stream, x)
    with _allocating(stream):
        if mine:
            out = x.new_empty((T, H))
        ws = _workspace(workspace, L.geg_moe_layer_workspace_bytes(T, k, I), x.device, None, check_errors)
    f = L.gnf4_moe_layer if nf4 else L.gmxfp4_moe_layer
    _check(f(x.data_ptr(), topk_ids.data_ptr(), topk_weights.data_ptr(), w13.data_ptr(), s13.data_ptr(), w2.data_ptr(),
             s2.data_ptr(), out.data_ptr(), T, k, H, I, E, ws.buf.data_ptr(), ws.buf.numel(),
             ctypes.byref(opts) if opts else None, raw))
    if mine:
        _outlive(stream, out)
    _check_device_errors(ws, check_errors, stream)
    return out


def gnf4_moe_layer(x, topk_ids, topk_weights, w13, absmax13, w2, absmax2, out=None,
                   workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                   check_errors: bool = False):
    """The routed experts of a whole MoE layer for a few tokens (T <= 16, T * k <= 256), in
    two launches: x bf16 [T, H], topk_ids int32 [T, k] and topk_weights fp32 [T, k] (as
    route_topk returns them), NF4 weights as gnf4_expert_block takes them -> out bf16
    [T, H] = sum over slots of weight * down(silu(gate) * up). Larger batches:
    route_sort, gnf4_expert_block, route_combine."""
    return _moe_layer(True, x, topk_ids, topk_weights, w13, absmax13, w2, absmax2, out, workspace, opts, stream,
                      check_errors)


def gmxfp4_moe_layer(x, topk_ids, topk_weights, blocks13, scales13, blocks2, scales2, out=None,
                     workspace: Workspace | None = None, opts: Opts | None = None, stream=None,
                     check_errors: bool = False):
    """The same layer on MXFP4 weights as gmxfp4_expert_block takes them."""
    if blocks13.dim() == 4:
        blocks13 = blocks13.reshape(blocks13.shape[0], blocks13.shape[1], -1)
    if blocks2.dim() == 4:
        blocks2 = blocks2.reshape(blocks2.shape[0], blocks2.shape[1], -1)
    return _moe_layer(False, x, topk_ids, topk_weights, blocks13, scales13, blocks2, scales2, out, workspace, opts,
                      stream, check_errors)


def _make_router_gate():
    import torch

    class RouterGate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k, renormalize):
            weights, ids = route_topk(logits, k, renormalize)
            ctx.save_for_backward(logits, ids, weights)
            ctx.renormalize = renormalize
            ctx.mark_non_differentiable(ids)
            return weights, ids

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dweights, _):
            logits, ids, weights = ctx.saved_tensors
            return route_topk_grad(dweights.contiguous(), logits, ids, weights, ctx.renormalize), None, None

    return RouterGate


def _make_dispatch_rows():
    import torch

    class DispatchRows(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, topk_ids, E):
            sizes, row_of, src_of, xs = route_sort(topk_ids, E, x)
            ctx.save_for_backward(row_of)
            ctx.k = topk_ids.shape[1]
            ctx.mark_non_differentiable(sizes, row_of, src_of)
            return xs, sizes, row_of, src_of

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dxs, *_):
            row_of, = ctx.saved_tensors
            return route_combine(dxs.contiguous(), row_of, None, ctx.k), None, None

    return DispatchRows


def _make_combine_rows():
    import torch

    class CombineRows(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, weights, row_of, src_of):
            ctx.save_for_backward(y, weights, row_of, src_of)
            return route_combine(y, row_of, weights, weights.shape[1])

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            y, weights, row_of, src_of = ctx.saved_tensors
            dy, dw = route_combine_grad(dout.contiguous(), y, row_of, weights, src_of)
            return dy, dw, None, None

    return CombineRows


_RouterGate = _LazyFn(_make_router_gate)
_DispatchRows = _LazyFn(_make_dispatch_rows)
_CombineRows = _LazyFn(_make_combine_rows)


def router_gate(logits, k: int, renormalize: bool = True):
    """route_topk as a torch autograd op: (weights fp32 [T, k], ids int32 [T, k]), the
    weights differentiable with respect to the logits."""
    return _RouterGate.apply(logits, int(k), bool(renormalize))


def dispatch_rows(x, topk_ids, E: int):
    """route_sort with the gather as a torch autograd op: x bf16 [T, H] -> (x_sorted bf16
    [T*k, H], sizes, row_of, src_of); the backward adds each token's k rows."""
    return _DispatchRows.apply(x, topk_ids, int(E))


def combine_rows(y, weights, row_of, src_of):
    """route_combine as a torch autograd op, differentiable with respect to the expert
    outputs y bf16 [T*k, N] and the router weights fp32 [T, k]."""
    return _CombineRows.apply(y, weights, row_of, src_of)


# ----------------------------------------------------------------------------- 16-bit grouped products
def _dtype16(t, name):
    code = _dtype(t, name)
    if code == 2:
        raise GegError(2, f"{name}: expected a bfloat16 or float16 tensor, got {t.dtype}")
    return code


def _dense(fn_name, x, xname, sizes, w, out, oname, width, zero_rest, workspace, opts, stream, check_errors):
    """Forward (x = a, out [M, N]) or gradient of the activations (x = dy, out [M, K])."""
    import torch
    dt = _dtype16(x, xname)
    if x.dim() != 2 or w.dim() != 3:
        raise GegError(2, f"{xname}: expected a 2-D tensor, w [E, N, K]")
    M = x.shape[0]
    E, N, K = w.shape
    _check_tensor(x, xname, x.dtype, (M, N + K - width))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_tensor(w, "w", x.dtype, (E, N, K))
    _check_tensor(out, oname, x.dtype, (M, width))
    _on_device(x, sizes, w, out)
    mine = out is None
    raw = _raw_stream(stream, x)
    with _allocating(stream):
        if mine:
            out = x.new_empty((M, width))
        ws = _workspace(workspace, lib().geg_grouped_workspace_bytes(int(fn_name == "geg_grouped_dgrad"), M, N, K, E), x.device,
                        None, check_errors)
    _check(getattr(lib(), fn_name)(x.data_ptr(), sizes.data_ptr(), w.data_ptr(), out.data_ptr(), dt, M, N, K, E,
                                   int(zero_rest), ws.buf.data_ptr(), ws.buf.numel(),
                                   ctypes.byref(opts) if opts else None, raw))
    if mine:
        _outlive(stream, out)
    _check_device_errors(ws, check_errors, stream)
    return out


def grouped_gemm(a, sizes, w, out=None, zero_rest: bool = False, workspace: Workspace | None = None,
                 opts: Opts | None = None, stream=None, check_errors: bool = False):
    """The grouped expert product with 16-bit weights: a [M, K] (bf16 or fp16, rows grouped
    by expert), sizes int32 [E], w [E, N, K] of a's type -> out [M, N] = a_e W_e^T, summed
    in fp32. K % 8 == 0. Rows past sum(sizes) stay as they were allocated, or are set to 0
    with zero_rest."""
    return _dense("geg_grouped_gemm", a, "a", sizes, w, out, "out", w.shape[1] if w.dim() == 3 else 0, zero_rest,
                  workspace, opts, stream, check_errors)


def grouped_dgrad(dy, sizes, w, dx=None, zero_rest: bool = False, workspace: Workspace | None = None,
                  opts: Opts | None = None, stream=None, check_errors: bool = False):
    """Gradient of grouped_gemm's activations: dy [M, N], w [E, N, K] -> dx [M, K] = dy_e W_e.
    N % 8 == 0 and K % 8 == 0."""
    return _dense("geg_grouped_dgrad", dy, "dy", sizes, w, dx, "dx", w.shape[2] if w.dim() == 3 else 0, zero_rest,
                  workspace, opts, stream, check_errors)


def grouped_wgrad(dy, a, sizes, dw=None, dtype=None, workspace: Workspace | None = None, opts: Opts | None = None,
                  stream=None, check_errors: bool = False):
    """Gradient of grouped_gemm's weights: dy [M, N], a [M, K], sizes int32 [E] -> dw
    [E, N, K] = dy_e^T a_e (0 for experts without rows), in dtype: a's (None) or
    torch.float32. N % 8 == 0 and K % 8 == 0."""
    import torch
    dt = _dtype16(dy, "dy")
    if dy.dim() != 2 or a.dim() != 2 or sizes.dim() != 1:
        raise GegError(2, "dy: expected [M, N], a [M, K], sizes [E]")
    M, N = dy.shape
    K, E = a.shape[1], sizes.shape[0]
    if dtype is None:
        dtype = dw.dtype if dw is not None else dy.dtype
    if dtype not in (dy.dtype, torch.float32):
        raise GegError(2, f"dtype: expected {dy.dtype} or torch.float32, got {dtype}")
    _check_tensor(dy, "dy", dy.dtype, (M, N))
    _check_tensor(a, "a", dy.dtype, (M, K))
    _check_tensor(sizes, "sizes", torch.int32, (E,))
    _check_tensor(dw, "dw", dtype, (E, N, K))
    _on_device(dy, a, sizes, dw)
    mine = dw is None
    raw = _raw_stream(stream, dy)
    with _allocating(stream):
        if mine:
            dw = dy.new_empty((E, N, K), dtype=dtype)
        ws = _workspace(workspace, lib().geg_grouped_workspace_bytes(2, M, N, K, E), dy.device, None, check_errors)
    _check(lib().geg_grouped_wgrad(dy.data_ptr(), a.data_ptr(), sizes.data_ptr(), dw.data_ptr(), dt,
                                   2 if dtype is torch.float32 else dt, M, N, K, E, ws.buf.data_ptr(), ws.buf.numel(),
                                   ctypes.byref(opts) if opts else None, raw))
    if mine:
        _outlive(stream, dw)
    _check_device_errors(ws, check_errors, stream)
    return dw


def _make_grouped_matmul():
    import torch

    class GroupedMatmul(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, sizes, w, check_errors):
            ctx.save_for_backward(a, sizes, w)
            ctx.check_errors = check_errors
            return grouped_gemm(a, sizes, w, zero_rest=True, check_errors=check_errors)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            a, sizes, w = ctx.saved_tensors
            dy = dy.contiguous()
            da = dw = None
            if ctx.needs_input_grad[0]:
                da = grouped_dgrad(dy, sizes, w, zero_rest=True, check_errors=ctx.check_errors)
            if ctx.needs_input_grad[2]:
                dw = grouped_wgrad(dy, a, sizes, check_errors=ctx.check_errors)
            return da, None, dw, None

    return GroupedMatmul


_GroupedMatmul = _LazyFn(_make_grouped_matmul)


def grouped_matmul(a, sizes, w, check_errors: bool = False):
    """grouped_gemm as a torch autograd op, differentiable with respect to the activations a
    [M, K] and the weights w [E, N, K]: training of experts that are not quantised, next to
    router_gate, dispatch_rows and combine_rows. Rows past sum(sizes) (a padded batch) give
    0 and get 0."""
    return _GroupedMatmul.apply(a, sizes, w, bool(check_errors))


# ----------------------------------------------------------------------------- adapters of many requests
def _pitch(t, name, dtype, shape):
    """Row pitch of a 2-D tensor of contiguous rows (a slice of columns, say)."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or (shape[1] > 1 and t.stride(1) != 1) or \
            (shape[0] > 1 and t.stride(0) < shape[1]):
        raise GegError(2, f"{name}: expected a {dtype} tensor of shape {list(shape)} with contiguous rows, got "
                          f"{t.dtype} {list(t.shape)} of strides {list(t.stride())}")
    return t.stride(0) if shape[0] > 1 else shape[1]


def request_lora(y, x, ids, lora_a, lora_b, scales=None, out=None, workspace: Workspace | None = None, stream=None,
                 check_errors: bool = False):
    """Low-rank adapters of many requests beside a projection that they share: out [M, N] =
    y + scales[i] (x A_i^T) B_i^T with each row's own adapter i = ids[t], ids int32 [M] in any
    order (negative: none). y [M, N] (what the projection gave; None for zeros), x [M, K],
    lora_a [L, r, K] and lora_b [L, N, r] of one type, bf16 or fp16; scales fp32 [L] or None;
    r 8, 16, ..., 128. out=y adds in place. x, y and out may be slices of columns (rows that
    start at multiples of 16 bytes). For rows routed to experts with adapters of their own:
    ids = adapter * E + expert over lora_a [adapters * E, r, K]."""
    import torch
    dt = _dtype16(x, "x")
    if x.dim() != 2 or lora_a.dim() != 3 or lora_b.dim() != 3:
        raise GegError(2, "x: expected [M, K], lora_a [L, r, K], lora_b [L, N, r]")
    M, K = x.shape
    L, r = lora_a.shape[0], lora_a.shape[1]
    N = lora_b.shape[1]
    ldx = _pitch(x, "x", x.dtype, (M, K))
    ldy = 0 if y is None else _pitch(y, "y", x.dtype, (M, N))
    _check_tensor(ids, "ids", torch.int32, (M,))
    _check_tensor(lora_a, "lora_a", x.dtype, (L, r, K))
    _check_tensor(lora_b, "lora_b", x.dtype, (L, N, r))
    _check_tensor(scales, "scales", torch.float32, (L,))
    ldo = N if out is None else _pitch(out, "out", x.dtype, (M, N))
    _on_device(x, y, ids, lora_a, lora_b, scales, out)
    mine = out is None
    raw = _raw_stream(stream, x)
    lib_ = lib()
    with _allocating(stream):
        if mine:
            out = x.new_empty((M, N))
        ws = _workspace(workspace, lib_.geg_request_lora_workspace_bytes(M, K, L, r), x.device, None, check_errors)
    _check(lib_.geg_request_lora(_addr(y), ldy, x.data_ptr(), ldx, ids.data_ptr(), lora_a.data_ptr(), lora_b.data_ptr(),
                                 _addr(scales), out.data_ptr(), ldo, dt, M, N, K, L, r, ws.buf.data_ptr(), ws.buf.numel(),
                                 raw))
    if mine:
        _outlive(stream, out)
    _check_device_errors(ws, check_errors, stream)
    return out


# ----------------------------------------------------------------------------- dropout
def _seed(seed, offset):
    """(seed, offset, rng tensor or None) of a seed given as an int or as a device int64 tensor
    {seed, offset}, whose offset the given one is added to."""
    import torch
    if isinstance(seed, torch.Tensor):
        _check_tensor(seed, "seed", torch.int64, (2,))
        return 0, int(offset) & 0xFFFFFFFFFFFFFFFF, seed
    return int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFFFFFFFFFF, None


def philox_dropout(x, p: float, seed, offset: int = 0, residual=None, out=None, stream=None):
    """Dropout from a counter-based generator (Philox4x32-10), its mask never stored: out =
    [residual +] x / (1 - p) where value i's 16 random bits are at least round(65536 p), else
    [residual +] 0 (1 - p as those bits have it). The mask follows from seed, offset and i
    alone: the same call over a gradient drops the same values. seed: an int, or an int64
    tensor {seed, offset} on the device, whose offset `offset` is added to and which a captured
    call reads anew on every replay. bf16, fp16 or fp32; out may be x or residual."""
    dt = _dtype(x, "x")
    seed, offset, rng = _seed(seed, offset)
    if not x.is_contiguous():
        raise GegError(2, f"x: expected a contiguous tensor, got strides {list(x.stride())} of shape {list(x.shape)}")
    _check_tensor(residual, "residual", x.dtype, x.shape)
    _check_tensor(out, "out", x.dtype, x.shape)
    _on_device(x, residual, out, rng)
    mine = out is None
    if mine:
        with _allocating(stream):
            out = x.new_empty(x.shape)
    _check(lib().geg_dropout(x.data_ptr(), _addr(residual), out.data_ptr(), dt, x.numel(), float(p), seed, offset,
                             _addr(rng), _raw_stream(stream, x)))
    if mine:
        _outlive(stream, out)
    return out


def _make_dropout():
    import torch

    class Dropout(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, p, seed, offset, residual):
            ctx.p, ctx.offset = p, offset
            ctx.seed = None if isinstance(seed, torch.Tensor) else seed
            ctx.save_for_backward(*(() if ctx.seed is not None else (seed,)))
            return philox_dropout(x, p, seed, offset, residual)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            seed = ctx.seed if ctx.seed is not None else ctx.saved_tensors[0]
            dx = None
            if ctx.needs_input_grad[0]:
                dx = philox_dropout(dout.contiguous(), ctx.p, seed, ctx.offset)
            return dx, None, None, None, dout if ctx.needs_input_grad[4] else None

    return Dropout


_Dropout = _LazyFn(_make_dropout)


def dropout(x, p: float, seed, offset: int = 0, residual=None):
    """philox_dropout as a torch autograd op, differentiable with respect to x and the
    residual. A seed given as a tensor must keep its values until the backward pass is done
    (torch refuses the backward pass of one changed in place): layers of one step take
    different offsets, the next step's values are set after the backward pass."""
    return _Dropout.apply(x, float(p), seed, int(offset), residual)
