"""ctypes binding of liblstm.so (C ABI declared in include/liblstm.h).

Argument marshalling only: every step of the LSTM forward pass and BPTT runs
inside the library's CUDA kernels.  torch tensors are used for device memory
and for the current CUDA stream; nothing here computes on them.  When the
shared library is missing, every entry point raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblstm.so")

LSTM_OK = 0
LSTM_ERR_INVALID_ARG = 1
LSTM_ERR_UNSUPPORTED = 2
LSTM_ERR_WORKSPACE = 3
LSTM_ERR_CUDA = 4
LSTM_ERR_TIMEOUT = 5
LSTM_ERR_NOT_CORESIDENT = 6

ABI_VERSION = 103  # the liblstm.h this binding mirrors (100 * major + minor)
LSTM_F32 = 0
LSTM_BF16 = 1
LSTM_F16 = 2

EXPORTS = ("lstm_fwd_workspace_size", "lstm_bwd_workspace_size", "lstm_fwd_workspace_size_ex",
           "lstm_fwd_workspace_size_max", "lstm_fwd", "lstm_bwd",
           "lstm_fwd_ex", "lstm_bwd_ex", "lstm_stack_fwd_workspace_size",
           "lstm_stack_bwd_workspace_size", "lstm_stack_bwd_workspace_size_min",
           "lstm_stack_fwd", "lstm_stack_bwd",
           "lstm_embed_fwd", "lstm_embed_bwd_workspace_size", "lstm_embed_bwd",
           "lstm_gdr_fwd_workspace_size", "lstm_gdr_bwd_workspace_size", "lstm_gdr_fwd",
           "lstm_gdr_bwd",
           "lstm_logprob_fwd", "lstm_logprob_bwd",
           "lstm_status", "lstm_profile_begin", "lstm_profile_end", "lstm_launch_count",
           "lstm_strerror", "lstm_abi_version")

PHASES = ("input_proj", "fwd_recur", "bwd_recur", "dW", "db", "dx", "other")


class LstmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: liblstm status {code} ({strerror(code)})")


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("B", ctypes.c_int), ("I", ctypes.c_int),
                ("H", ctypes.c_int), ("dtype", ctypes.c_int)]


LSTM_DIR_FORWARD, LSTM_DIR_REVERSE = 0, 1
LSTM_GATES_IFJO, LSTM_GATES_IJFO = 0, 1
GATE_ORDERS = {"ifjo": LSTM_GATES_IFJO, "ijfo": LSTM_GATES_IJFO}


class Options(ctypes.Structure):
    """lstm_options: the seq_length mask (device pointer or None), the
    direction (LSTM_DIR_FORWARD / LSTM_DIR_REVERSE) and the gate_order
    (LSTM_GATES_IFJO / LSTM_GATES_IJFO)."""
    _fields_ = [("seq_mask", ctypes.c_void_p), ("direction", ctypes.c_int),
                ("gate_order", ctypes.c_int)]


class EmbedDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("vocab", ctypes.c_int), ("I", ctypes.c_int),
                ("dtype", ctypes.c_int), ("id_bytes", ctypes.c_int)]


class GdrDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "B", "Hk", "Hv", "K", "V", "dtype")] + \
        [(n, ctypes.c_longlong) for n in ("ldq", "ldk", "ldv")]


class GdrOptions(ctypes.Structure):
    """lstm_gdr_options: lengths [B] int32 (device pointer or None), scale."""
    _fields_ = [("lengths", ctypes.c_void_p), ("scale", ctypes.c_float)]


class LogprobDims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("vocab", ctypes.c_int), ("ld", ctypes.c_longlong),
                ("top", ctypes.c_int), ("dtype", ctypes.c_int), ("id_bytes", ctypes.c_int)]


_lib = None


def load(path: str = LIB_PATH):
    """Load liblstm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"liblstm.so not found at {path}: build it with "
                           "`python -m backward_lstm_fwd_b200.build`")
    lib = ctypes.CDLL(path)
    vp, sz, ip = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    dp = ctypes.POINTER(Dims)
    lib.lstm_fwd_workspace_size.argtypes = [dp]
    lib.lstm_fwd_workspace_size.restype = sz
    lib.lstm_bwd_workspace_size.argtypes = [dp]
    lib.lstm_bwd_workspace_size.restype = sz
    lib.lstm_fwd_workspace_size_max.argtypes = [dp]
    lib.lstm_fwd_workspace_size_max.restype = sz
    lib.lstm_fwd.argtypes = [dp] + [vp] * 10 + [vp, sz, vp]
    lib.lstm_fwd.restype = ip
    lib.lstm_bwd.argtypes = [dp] + [vp] * 15 + [vp, sz, vp]
    lib.lstm_bwd.restype = ip
    op = ctypes.POINTER(Options)
    lib.lstm_fwd_workspace_size_ex.argtypes = [dp, op]
    lib.lstm_fwd_workspace_size_ex.restype = sz
    lib.lstm_fwd_ex.argtypes = [dp, op] + [vp] * 10 + [vp, sz, vp]
    lib.lstm_fwd_ex.restype = ip
    lib.lstm_bwd_ex.argtypes = [dp, op] + [vp] * 15 + [vp, sz, vp]
    lib.lstm_bwd_ex.restype = ip
    pp = ctypes.POINTER(ctypes.c_void_p)  # host array of device pointers
    lib.lstm_stack_fwd_workspace_size.argtypes = [dp, ip]
    lib.lstm_stack_fwd_workspace_size.restype = sz
    lib.lstm_stack_bwd_workspace_size.argtypes = [dp, ip]
    lib.lstm_stack_bwd_workspace_size.restype = sz
    lib.lstm_stack_bwd_workspace_size_min.argtypes = [dp, ip]
    lib.lstm_stack_bwd_workspace_size_min.restype = sz
    lib.lstm_stack_fwd.argtypes = [dp, ip, op, vp, pp, pp] + [vp] * 7 + [vp, sz, vp]
    lib.lstm_stack_fwd.restype = ip
    lib.lstm_stack_bwd.argtypes = [dp, ip, op] + [vp] * 4 + [pp] + [vp] * 6 + [pp, pp] + \
        [vp] * 2 + [vp, sz, vp]
    lib.lstm_stack_bwd.restype = ip
    lib.lstm_status.argtypes = [vp, sz, vp]
    lib.lstm_status.restype = ip
    lib.lstm_strerror.argtypes = [ip]
    lib.lstm_strerror.restype = ctypes.c_char_p
    lib.lstm_abi_version.argtypes = []
    lib.lstm_abi_version.restype = ip
    lib.lstm_profile_begin.argtypes = []
    lib.lstm_profile_begin.restype = ip
    lib.lstm_profile_end.argtypes = [ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_longlong)]
    lib.lstm_profile_end.restype = ip
    lib.lstm_launch_count.argtypes = []
    lib.lstm_launch_count.restype = ctypes.c_longlong
    lib.lstm_fwd_noalloc.argtypes = [dp] + [vp] * 10 + [vp]
    lib.lstm_fwd_noalloc.restype = ip
    lib.lstm_fwd_noalloc_status.argtypes = [vp]
    lib.lstm_fwd_noalloc_status.restype = ip
    ll = ctypes.c_longlong
    lib.lstm_test_tc_gemm.argtypes = [ip, ip, ip, vp, ll, ip, vp, ll, ip, vp, vp, ll, vp, sz, vp]
    lib.lstm_test_tc_gemm.restype = ip
    lib.lstm_test_set_wait_fault.argtypes = [ip, ll]
    lib.lstm_test_set_wait_fault.restype = ip
    lib.lstm_test_last_paths.argtypes = [ctypes.POINTER(ip), ctypes.POINTER(ip)]
    lib.lstm_test_last_paths.restype = ip
    lib.lstm_test_last_stack_chunks.argtypes = [ctypes.POINTER(ip), ctypes.POINTER(ip)]
    lib.lstm_test_last_stack_chunks.restype = ip
    lib.lstm_test_last_persist_split.argtypes = [ctypes.POINTER(ip), ctypes.POINTER(ip)]
    lib.lstm_test_last_persist_split.restype = ip
    lib.lstm_test_bwd_chunks.argtypes = [ip]
    lib.lstm_test_bwd_chunks.restype = ip
    lib.lstm_test_chunk_bound.argtypes = [ip, ip, ip]
    lib.lstm_test_chunk_bound.restype = ip
    ep, lp, fp = ctypes.POINTER(EmbedDims), ctypes.POINTER(LogprobDims), ctypes.c_float
    lib.lstm_embed_fwd.argtypes = [ep, vp, vp, fp, vp, vp]
    lib.lstm_embed_fwd.restype = ip
    lib.lstm_embed_bwd_workspace_size.argtypes = [ep]
    lib.lstm_embed_bwd_workspace_size.restype = sz
    lib.lstm_embed_bwd.argtypes = [ep, vp, vp, fp, ip, vp, vp, sz, vp]
    lib.lstm_embed_bwd.restype = ip
    lib.lstm_logprob_fwd.argtypes = [lp, vp, vp, fp] + [vp] * 6
    lib.lstm_logprob_fwd.restype = ip
    lib.lstm_logprob_bwd.argtypes = [lp, vp, vp, fp] + [vp] * 5 + [ll, vp]
    lib.lstm_logprob_bwd.restype = ip
    gp, go = ctypes.POINTER(GdrDims), ctypes.POINTER(GdrOptions)
    lib.lstm_gdr_fwd_workspace_size.argtypes = [gp, ip]
    lib.lstm_gdr_fwd_workspace_size.restype = sz
    lib.lstm_gdr_bwd_workspace_size.argtypes = [gp]
    lib.lstm_gdr_bwd_workspace_size.restype = sz
    lib.lstm_gdr_fwd.argtypes = [gp, go] + [vp] * 10 + [vp, sz, vp]
    lib.lstm_gdr_fwd.restype = ip
    lib.lstm_gdr_bwd.argtypes = [gp, go] + [vp] * 16 + [vp, sz, vp]
    lib.lstm_gdr_bwd.restype = ip
    v = lib.lstm_abi_version()
    if v // 100 != ABI_VERSION // 100 or v < ABI_VERSION:
        raise RuntimeError(f"{path}: ABI version {v}, this binding needs {ABI_VERSION} "
                           "(rebuild with `python -m backward_lstm_fwd_b200.build`)")
    if path == LIB_PATH:
        _lib = lib
    return lib


def strerror(code: int) -> str:
    try:
        return load().lstm_strerror(int(code)).decode()
    except RuntimeError:
        return "liblstm not loaded"


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return LSTM_F32
    if dt == torch.bfloat16:
        return LSTM_BF16
    if dt == torch.float16:
        return LSTM_F16
    raise ValueError(f"unsupported compute dtype {dt}")


def dims(T: int, B: int, I: int, H: int, dtype) -> Dims:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return Dims(int(T), int(B), int(I), int(H), code)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr() if t.numel() > 0 else None


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def fwd_workspace_size(d: Dims, mask=None, reverse: bool = False, gate_order="ifjo") -> int:
    """Forward workspace bytes for the plan this call takes on the current
    device (lstm_fwd_workspace_size, or _ex with the call's options)."""
    if _plain(mask, reverse, gate_order):
        return int(load().lstm_fwd_workspace_size(ctypes.byref(d)))
    opt = _options(mask, reverse, gate_order)
    return int(load().lstm_fwd_workspace_size_ex(ctypes.byref(d), ctypes.byref(opt)))


def fwd_workspace_size_max(d: Dims) -> int:
    """Forward workspace bytes that cover every plan on every device."""
    return int(load().lstm_fwd_workspace_size_max(ctypes.byref(d)))


def bwd_workspace_size(d: Dims) -> int:
    return int(load().lstm_bwd_workspace_size(ctypes.byref(d)))


def _gate_order(gate_order) -> int:
    """"ifjo" / "ijfo" (the attribute's values) or the C constant itself."""
    return GATE_ORDERS[gate_order] if isinstance(gate_order, str) else int(gate_order)


def _options(mask, reverse, gate_order):
    return Options(_p(mask), LSTM_DIR_REVERSE if reverse else LSTM_DIR_FORWARD,
                   _gate_order(gate_order))


def _plain(mask, reverse, gate_order) -> bool:
    return mask is None and not reverse and _gate_order(gate_order) == LSTM_GATES_IFJO


def lstm_fwd(d: Dims, x, W, b, h0, c0, y, hT, cT, gates, cells, ws, ws_bytes=None,
             stream=None, check: bool = True, mask=None, reverse: bool = False,
             gate_order="ifjo") -> int:
    """Direct call of the C entry point lstm_fwd, or lstm_fwd_ex with a
    variable-length mask [T,B,H] (1 = real step, 0 = padding), the reverse
    direction and / or gate_order "ijfo" (device tensors or raw pointers)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    if _plain(mask, reverse, gate_order):
        rc = load().lstm_fwd(ctypes.byref(d), _p(x), _p(W), _p(b), _p(h0), _p(c0), _p(y),
                             _p(hT), _p(cT), _p(gates), _p(cells), _p(ws), ws_bytes,
                             _stream(stream))
    else:
        opt = _options(mask, reverse, gate_order)
        rc = load().lstm_fwd_ex(ctypes.byref(d), ctypes.byref(opt), _p(x), _p(W), _p(b), _p(h0),
                                _p(c0), _p(y), _p(hT), _p(cT), _p(gates), _p(cells), _p(ws),
                                ws_bytes, _stream(stream))
    if check and rc != LSTM_OK:
        raise LstmError(rc, "lstm_fwd")
    return rc


def lstm_bwd(d: Dims, dy, dhT, dcT, x, W, h0, c0, y, gates, cells, dx, dW, db, dh0, dc0, ws,
             ws_bytes=None, stream=None, check: bool = True, mask=None,
             reverse: bool = False, gate_order="ifjo") -> int:
    """Direct call of the C entry point lstm_bwd, or lstm_bwd_ex with the
    forward's mask, direction and gate_order (device tensors or raw pointers)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    if _plain(mask, reverse, gate_order):
        rc = load().lstm_bwd(ctypes.byref(d), _p(dy), _p(dhT), _p(dcT), _p(x), _p(W), _p(h0),
                             _p(c0), _p(y), _p(gates), _p(cells), _p(dx), _p(dW), _p(db),
                             _p(dh0), _p(dc0), _p(ws), ws_bytes, _stream(stream))
    else:
        opt = _options(mask, reverse, gate_order)
        rc = load().lstm_bwd_ex(ctypes.byref(d), ctypes.byref(opt), _p(dy), _p(dhT), _p(dcT),
                                _p(x), _p(W), _p(h0), _p(c0), _p(y), _p(gates), _p(cells),
                                _p(dx), _p(dW), _p(db), _p(dh0), _p(dc0), _p(ws), ws_bytes,
                                _stream(stream))
    if check and rc != LSTM_OK:
        raise LstmError(rc, "lstm_bwd")
    return rc


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def _ptr_array(ts):
    """A host array of device pointers (None, a tensor or an int per entry);
    None for no array at all."""
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[_p(t) for t in ts])


def stack_fwd_workspace_size(d: Dims, L: int) -> int:
    return int(load().lstm_stack_fwd_workspace_size(ctypes.byref(d), int(L)))


def stack_bwd_workspace_size(d: Dims, L: int) -> int:
    return int(load().lstm_stack_bwd_workspace_size(ctypes.byref(d), int(L)))


def stack_bwd_workspace_size_min(d: Dims, L: int) -> int:
    """The smallest workspace lstm_stack_bwd accepts (layers one after another)."""
    return int(load().lstm_stack_bwd_workspace_size_min(ctypes.byref(d), int(L)))


def lstm_stack_fwd(d: Dims, L: int, x, Ws, bs, h0, c0, y, hT, cT, gates, cells, ws,
                   ws_bytes=None, stream=None, check: bool = True, mask=None,
                   reverse: bool = False, gate_order="ifjo") -> int:
    """Direct call of lstm_stack_fwd: Ws / bs are lists of L device tensors
    (bs may be None); the [L][...] arrays are single tensors."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    opt = _options(mask, reverse, gate_order)
    Wa, ba = _ptr_array(Ws), _ptr_array(bs)
    rc = load().lstm_stack_fwd(ctypes.byref(d), int(L), ctypes.byref(opt), _p(x), Wa, ba, _p(h0),
                               _p(c0), _p(y), _p(hT), _p(cT), _p(gates), _p(cells), _p(ws),
                               ws_bytes, _stream(stream))
    if check and rc != LSTM_OK:
        raise LstmError(rc, "lstm_stack_fwd")
    return rc


def lstm_stack_bwd(d: Dims, L: int, dy, dhT, dcT, x, Ws, h0, c0, y, gates, cells, dx, dWs, dbs,
                   dh0, dc0, ws, ws_bytes=None, stream=None, check: bool = True, mask=None,
                   reverse: bool = False, gate_order="ifjo") -> int:
    """Direct call of lstm_stack_bwd: Ws, dWs and dbs are lists of L device
    tensors."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    opt = _options(mask, reverse, gate_order)
    Wa, dWa, dba = _ptr_array(Ws), _ptr_array(dWs), _ptr_array(dbs)
    rc = load().lstm_stack_bwd(ctypes.byref(d), int(L), ctypes.byref(opt), _p(dy), _p(dhT),
                               _p(dcT), _p(x), Wa, _p(h0), _p(c0), _p(y), _p(gates), _p(cells),
                               _p(dx), dWa, dba, _p(dh0), _p(dc0), _p(ws), ws_bytes,
                               _stream(stream))
    if check and rc != LSTM_OK:
        raise LstmError(rc, "lstm_stack_bwd")
    return rc


def lstm_fwd_noalloc(d: Dims, x, W, b, h0, c0, y, hT, cT, gates, cells, stream=None,
                     check: bool = True) -> int:
    """Direct call of lstm_fwd_noalloc: lstm_fwd with the library's static
    device scratch instead of a caller workspace (for callers that may not
    allocate device memory)."""
    rc = load().lstm_fwd_noalloc(ctypes.byref(d), _p(x), _p(W), _p(b), _p(h0), _p(c0), _p(y),
                                 _p(hT), _p(cT), _p(gates), _p(cells), _stream(stream))
    if check and rc != LSTM_OK:
        raise LstmError(rc, "lstm_fwd_noalloc")
    return rc


def lstm_fwd_noalloc_status(stream=None) -> int:
    """Synchronise `stream`, then read and clear the status word of the static
    scratch lstm_fwd_noalloc uses on the current device."""
    return int(load().lstm_fwd_noalloc_status(_stream(stream)))


def lstm_status(ws, ws_bytes=None, stream=None) -> int:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    return int(load().lstm_status(_p(ws), ws_bytes, _stream(stream)))


def profile_begin() -> None:
    load().lstm_profile_begin()


def profile_end():
    """Per-phase (device ms, kernel launches) since profile_begin()."""
    n = len(PHASES)
    ms = (ctypes.c_double * n)()
    la = (ctypes.c_longlong * n)()
    rc = load().lstm_profile_end(ms, la)
    if rc != LSTM_OK:
        raise LstmError(rc, "lstm_profile_end")
    return {p: (ms[i], la[i]) for i, p in enumerate(PHASES)}


def launch_count() -> int:
    return int(load().lstm_launch_count())


def test_tc_gemm(M, N, K, A, lda, a_mn_major, Bm, ldb, b_mn_major, bias, C, ldc, ws,
                 stream=None) -> int:
    """Test hook (include/liblstm_testing.h): C = A B^T (+ bias) on the tcgen05 core."""
    return int(load().lstm_test_tc_gemm(M, N, K, _p(A), lda, a_mn_major, _p(Bm), ldb, b_mn_major,
                                         _p(bias), _p(C), ldc, _p(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)))


def test_set_wait_fault(skip_cta: int, wait_ns: int) -> None:
    """Test hook: CTA `skip_cta` of persistent launches never arrives (-1: off);
    device-side waits give up after wait_ns (<= 0: default 2 s)."""
    load().lstm_test_set_wait_fault(int(skip_cta), int(wait_ns))


def test_last_paths():
    """Test hook: (forward, backward) recurrent kernel of the last calls:
    0 per-step CUDA cores, 1 persistent K-resident, 2 persistent cluster."""
    f, b = ctypes.c_int(), ctypes.c_int()
    load().lstm_test_last_paths(ctypes.byref(f), ctypes.byref(b))
    return f.value, b.value


def test_last_stack_chunks():
    """Test hook: (forward, backward) chunks per layer of the last stack calls'
    layer wavefronts (0: layer after layer; -1: no such call yet)."""
    f, b = ctypes.c_int(), ctypes.c_int()
    load().lstm_test_last_stack_chunks(ctypes.byref(f), ctypes.byref(b))
    return f.value, b.value


def test_last_persist_split():
    """Test hook: (forward, backward) cluster size of the last persistent
    CUDA-core recurrences (0: none yet)."""
    f, b = ctypes.c_int(), ctypes.c_int()
    load().lstm_test_last_persist_split(ctypes.byref(f), ctypes.byref(b))
    return f.value, b.value


# ------------------------------------------------------------------ helpers
def empty_workspace(nbytes: int, device) -> torch.Tensor:
    """A byte tensor usable as workspace (torch's allocator returns 256-byte
    aligned blocks)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class State:
    """Outputs of one forward call (device tensors), kept for the backward."""

    def __init__(self, T, B, I, H, cd, device):
        self.dims = dims(T, B, I, H, cd)
        self.y = torch.empty((T, B, H), dtype=cd, device=device)
        self.hT = torch.empty((B, H), dtype=cd, device=device)
        self.cT = torch.empty((B, H), dtype=torch.float32, device=device)
        self.gates = torch.empty((T, B, 4 * H), dtype=cd, device=device)
        self.cells = torch.empty((T, B, H), dtype=torch.float32, device=device)


class Grads:
    def __init__(self, T, B, I, H, device):
        f = torch.float32
        self.dx = torch.empty((T, B, I), dtype=f, device=device)
        self.dW = torch.empty((4 * H, H + I), dtype=f, device=device)
        self.db = torch.empty((4 * H,), dtype=f, device=device)
        self.dh0 = torch.empty((B, H), dtype=f, device=device)
        self.dc0 = torch.empty((B, H), dtype=f, device=device)


def forward(x, W, b=None, h0=None, c0=None, ws=None, stream=None, mask=None,
            reverse: bool = False, gate_order="ifjo") -> State:
    """Allocate outputs and run lstm_fwd (lstm_fwd_ex with a mask, the
    reverse direction or gate_order "ijfo").  x [T,B,I], W [4H,H+I] and mask [T,B,H] share the
    compute dtype (float32 or bfloat16); c0 is float32."""
    T, B, I = x.shape
    H = W.shape[0] // 4
    st = State(T, B, I, H, x.dtype, x.device)
    if ws is None:
        ws = empty_workspace(fwd_workspace_size(st.dims, mask, reverse, gate_order), x.device)
    lstm_fwd(st.dims, x, W, b, h0, c0, st.y, st.hT, st.cT, st.gates, st.cells, ws, stream=stream,
             mask=mask, reverse=reverse, gate_order=gate_order)
    return st


def backward(st: State, x, W, h0=None, c0=None, dy=None, dhT=None, dcT=None, ws=None,
             stream=None, mask=None, reverse: bool = False, gate_order="ifjo") -> Grads:
    """Allocate gradients and run lstm_bwd on the saved state of forward()
    (lstm_bwd_ex with the forward's mask, direction and gate_order)."""
    T, B, I = x.shape
    H = W.shape[0] // 4
    g = Grads(T, B, I, H, x.device)
    if ws is None:
        ws = empty_workspace(bwd_workspace_size(st.dims), x.device)
    lstm_bwd(st.dims, dy, dhT, dcT, x, W, h0, c0, st.y, st.gates, st.cells, g.dx, g.dW, g.db,
             g.dh0, g.dc0, ws, stream=stream, mask=mask, reverse=reverse,
             gate_order=gate_order)
    return g


class StackState:
    """Outputs of one lstm_stack_fwd call: every layer's saved state."""

    def __init__(self, L, T, B, I, H, cd, device):
        self.L = L
        self.dims = dims(T, B, I, H, cd)
        self.y = torch.empty((L, T, B, H), dtype=cd, device=device)
        self.hT = torch.empty((L, B, H), dtype=cd, device=device)
        self.cT = torch.empty((L, B, H), dtype=torch.float32, device=device)
        self.gates = torch.empty((L, T, B, 4 * H), dtype=cd, device=device)
        self.cells = torch.empty((L, T, B, H), dtype=torch.float32, device=device)


class StackGrads:
    def __init__(self, L, T, B, I, H, device):
        f = torch.float32
        self.dx = torch.empty((T, B, I), dtype=f, device=device)
        self.dW = [torch.empty((4 * H, H + (I if l == 0 else H)), dtype=f, device=device)
                   for l in range(L)]
        self.db = [torch.empty((4 * H,), dtype=f, device=device) for _ in range(L)]
        self.dh0 = torch.empty((L, B, H), dtype=f, device=device)
        self.dc0 = torch.empty((L, B, H), dtype=f, device=device)


def forward_stack(x, Ws, bs=None, h0=None, c0=None, ws=None, stream=None, mask=None,
                  reverse: bool = False, gate_order="ifjo") -> StackState:
    """Allocate outputs and run lstm_stack_fwd.  x [T,B,I]; Ws[l] [4H, H+I_l];
    h0 [L,B,H] (compute dtype), c0 [L,B,H] float32."""
    T, B, I = x.shape
    L, H = len(Ws), Ws[0].shape[0] // 4
    st = StackState(L, T, B, I, H, x.dtype, x.device)
    if ws is None:
        ws = empty_workspace(stack_fwd_workspace_size(st.dims, L), x.device)
    lstm_stack_fwd(st.dims, L, x, Ws, bs, h0, c0, st.y, st.hT, st.cT, st.gates, st.cells, ws,
                   stream=stream, mask=mask, reverse=reverse, gate_order=gate_order)
    return st


def backward_stack(st: StackState, x, Ws, h0=None, c0=None, dy=None, dhT=None, dcT=None,
                   ws=None, stream=None, mask=None, reverse: bool = False,
                   gate_order="ifjo") -> StackGrads:
    """Allocate gradients and run lstm_stack_bwd on the saved state of
    forward_stack()."""
    T, B, I = x.shape
    L, H = len(Ws), Ws[0].shape[0] // 4
    g = StackGrads(L, T, B, I, H, x.device)
    if ws is None:
        ws = empty_workspace(stack_bwd_workspace_size(st.dims, L), x.device)
    lstm_stack_bwd(st.dims, L, dy, dhT, dcT, x, Ws, h0, c0, st.y, st.gates, st.cells, g.dx, g.dW,
                   g.db, g.dh0, g.dc0, ws, stream=stream, mask=mask, reverse=reverse,
                   gate_order=gate_order)
    return g


# ------------------------------------------- operators of a language model
LOGPROB_MAX_TOP = 64


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on(ref: torch.Tensor, **ts) -> None:
    """Every tensor given is on ref's CUDA device."""
    if not ref.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    dev = ref.get_device()
    for name, t in ts.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on another device")


def _flat(ref: torch.Tensor, **ts) -> None:
    """Every tensor given is contiguous and on ref's CUDA device."""
    if not ref.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    dev = ref.get_device()
    for name, t in ts.items():
        if t is not None:
            if t.get_device() != dev:
                raise ValueError(f"{name} is on another device")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")


def _shaped(t: Optional[torch.Tensor], name: str, shape, dtype=None) -> None:
    if t is not None:
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, want {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name}: {t.dtype}, want {dtype}")


def _workspace(like: torch.Tensor, nbytes: int) -> torch.Tensor:
    """empty_workspace() beside a tensor."""
    return like.new_empty(max(nbytes, 256), dtype=torch.uint8)


def _sizes(*n: int) -> None:
    if max(n) >= 1 << 31:
        raise ValueError(f"sizes {n}: each must be below 2**31")


def _id_bytes(ids: Optional[torch.Tensor]) -> int:
    if ids is None or ids.dtype == torch.int64:
        return 8
    if ids.dtype != torch.int32:
        raise ValueError(f"token ids must be int32 or int64, not {ids.dtype}")
    return 4


def _run(code: int, where: str) -> None:
    if code != LSTM_OK:
        raise LstmError(code, where)


def _ws_bytes(ws: torch.Tensor) -> int:
    return ws.numel() * ws.element_size()


def _at(t: Optional[torch.Tensor]):
    """Device pointer of a tensor that may be absent or empty."""
    return (t.data_ptr() or None) if t is not None else None


def _elsewhere(t: torch.Tensor, stream) -> bool:
    """The call belongs on another device or stream than the current ones."""
    return stream is not None or torch.cuda.current_device() != t.get_device()


def _there(t: torch.Tensor, stream, *used):
    """Context that makes the tensor's device current, or a stream of it: what
    a call allocates then belongs to the stream it works on.  The tensors that
    a given stream uses are known to the allocator: their memory is not reused
    before the call is done, even if the caller lets go of them at once."""
    if stream is None:
        return torch.cuda.device(t.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=t.device)
    _need(stream.device == t.device, "stream is on another device")
    for u in (t, *used):
        if u is not None:
            u.record_stream(stream)
    return torch.cuda.stream(stream)


def _used_here(*kept) -> None:
    """What a forward kept is used on another stream than it was made on."""
    for u in kept:
        if u is not None:
            u.record_stream(torch.cuda.current_stream(u.device))


def _here(t: torch.Tensor) -> int:
    """The current stream of the tensor's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def embed_dims(N: int, vocab: int, I: int, dtype, id_bytes: int = 8) -> EmbedDims:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return EmbedDims(int(N), int(vocab), int(I), code, int(id_bytes))


def embed(ids, table, scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """lstm_embed_fwd: x[..., I] = scale * table[ids] (table [vocab, I], ids
    int32 / int64 of any shape, e.g. [T, B] for an x [T, B, I]); ids outside
    the table are padding and give zeros."""
    _need(table.dim() == 2, "table must be [vocab, I]")
    _flat(table, table=table, ids=ids, out=out)
    vocab, I = table.shape
    N, shape = ids.numel(), (*ids.shape, I)
    _sizes(N, vocab, I)
    _shaped(out, "out", shape, table.dtype)
    if _elsewhere(table, stream):
        with _there(table, stream, ids, out):
            return embed(ids, table, scale, out)
    if out is None:
        out = table.new_empty(*shape)
    d = EmbedDims(N, vocab, I, dtype_code(table.dtype), _id_bytes(ids))
    _run(load().lstm_embed_fwd(ctypes.byref(d), _at(ids), _at(table), float(scale), _at(out),
                               _here(table)), "lstm_embed_fwd")
    return out


def embed_bwd_workspace_size(d: EmbedDims) -> int:
    return int(load().lstm_embed_bwd_workspace_size(ctypes.byref(d)))


def embed_backward(ids, dx, vocab: int, scale: float = 1.0, out=None, accumulate: bool = False,
                   ws=None, stream=None) -> torch.Tensor:
    """lstm_embed_bwd: the table's gradient [vocab, I] (float32) of
    embed(ids, table, scale) for dx [..., I] (float32, bfloat16 or float16).
    accumulate adds to `out` instead of overwriting it."""
    I = dx.shape[-1]
    _flat(dx, ids=ids, dx=dx, out=out, ws=ws)
    _shaped(dx, "dx", (*ids.shape, I))
    _need(not accumulate or out is not None, "accumulate needs out")
    N = ids.numel()
    _sizes(N, vocab, I)
    _shaped(out, "out", (vocab, I), torch.float32)
    if _elsewhere(dx, stream):
        with _there(dx, stream, ids, out, ws):
            return embed_backward(ids, dx, vocab, scale, out, accumulate, ws)
    if out is None:
        out = dx.new_empty(vocab, I, dtype=torch.float32)
    d = EmbedDims(N, vocab, I, dtype_code(dx.dtype), _id_bytes(ids))
    if ws is None:
        ws = _workspace(dx, embed_bwd_workspace_size(d))
    _run(load().lstm_embed_bwd(ctypes.byref(d), _at(ids), _at(dx), float(scale), int(accumulate),
                               _at(out), _at(ws), _ws_bytes(ws), _here(dx)), "lstm_embed_bwd")
    return out


class LogProbs:
    """Outputs of one logprobs() call (float32; top_ids int32), kept for the
    backward.  logp is None without targets, top_ids / top_logp with top = 0."""

    def __init__(self, N, top, has_targets, inv_temp, logits, made_on):
        self.inv_temp, self.made_on = inv_temp, made_on  # (a raw stream)
        self.vocab = logits.shape[1]
        # one allocation: rows of N for stats (2), entropy and logp, then top_logp and top_ids
        self._buf = buf = logits.new_empty(4 + 2 * top, N, dtype=torch.float32)
        self.entropy = buf[2]
        self.logp = buf[3] if has_targets else None
        self.top_logp = self.top_ids = None
        if top:
            self.top_logp = buf.as_strided((N, top), (top, 1), 4 * N)
            self.top_ids = buf.view(torch.int32).as_strided((N, top), (top, 1), (4 + top) * N)

    @property
    def stats(self) -> torch.Tensor:
        """[N, 2]: the row's largest logit and log2 sum 2^(c (x - largest)), c =
        log2(e) / temperature."""
        return self._buf[:2].view(-1, 2)

    @property
    def lse(self) -> torch.Tensor:
        """log sum exp(logits / temperature) of every row."""
        return self.stats[:, 0] * self.inv_temp + self.stats[:, 1] * math.log(2.0)


def logprob_dims(N: int, vocab: int, dtype, ld: Optional[int] = None, top: int = 0,
                 id_bytes: int = 8) -> LogprobDims:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return LogprobDims(int(N), int(vocab), int(vocab if ld is None else ld), int(top), code,
                       int(id_bytes))


def _rows(t: torch.Tensor, name: str) -> int:
    """Row stride of a [N, vocab] tensor whose rows are dense."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [N, vocab]")
    N, vocab = t.shape
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be dense")
    _sizes(N, vocab)
    ld = t.stride(0) if N > 1 else vocab
    if ld < vocab:
        raise ValueError(f"{name}: rows overlap")
    return ld


def logprobs(logits, targets=None, top: int = 0, temperature: float = 1.0,
             stream=None) -> LogProbs:
    """lstm_logprob_fwd on logits [N, vocab] (dense rows, any row stride):
    log-probability of targets [N], entropy, and the `top` best alternatives
    of every row at softmax(logits / temperature)."""
    ld = _rows(logits, "logits")
    N, vocab = logits.shape
    _flat(logits, targets=targets)
    _shaped(targets, "targets", (N,))
    _need(temperature > 0, "temperature must be positive")
    if not 0 <= top <= LOGPROB_MAX_TOP:  # (before the outputs are allocated)
        raise LstmError(LSTM_ERR_INVALID_ARG if top < 0 else LSTM_ERR_UNSUPPORTED, "lstm_logprob_fwd")
    if _elsewhere(logits, stream):
        with _there(logits, stream, targets):
            return logprobs(logits, targets, top, temperature)
    here = _here(logits)
    st = LogProbs(N, top, targets is not None, 1.0 / temperature, logits, here)
    d = LogprobDims(N, vocab, ld, top, dtype_code(logits.dtype), _id_bytes(targets))
    _run(load().lstm_logprob_fwd(ctypes.byref(d), _at(logits), _at(targets), st.inv_temp,
                                 _at(st.logp), _at(st.entropy), _at(st._buf), _at(st.top_ids),
                                 _at(st.top_logp), here), "lstm_logprob_fwd")
    return st


def logprobs_backward(st: LogProbs, logits, targets=None, dlogp=None, dentropy=None,
                      temperature: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """lstm_logprob_bwd: the gradient [N, vocab] of the logits, in their type; out
    may be logits.  Without `out` it has their row stride where that is the
    vocabulary and some padding (rows cut from a wider tensor lie close)."""
    ld = _rows(logits, "logits")
    N, vocab = logits.shape
    _flat(logits, targets=targets, dlogp=dlogp, dentropy=dentropy, state=st.entropy)
    _on(logits, out=out)
    _shaped(targets, "targets", (N,))
    _shaped(dlogp, "dlogp", (N,), torch.float32)
    _shaped(dentropy, "dentropy", (N,), torch.float32)
    _shaped(st.entropy, "the state's entropy", (N,))
    _shaped(out, "out", (N, vocab), logits.dtype)
    _need(1.0 / temperature == st.inv_temp, "temperature differs from the forward's")
    _need(vocab == st.vocab, "the state belongs to a forward of another vocabulary")
    if _elsewhere(logits, stream):
        with _there(logits, stream, targets, dlogp, dentropy, out):
            return logprobs_backward(st, logits, targets, dlogp, dentropy, temperature, out)
    here = _here(logits)
    if here != st.made_on:
        _used_here(st._buf)
    ldd = ld
    if out is not None:
        ldd = _rows(out, "out")
    else:
        if ld - vocab > max(64, vocab // 8):  # closer, with rows that still start alike modulo 16 bytes
            ldd = vocab + (ld - vocab) % (16 // logits.element_size())
        out = logits.new_empty(N, ldd)
        if ldd != vocab:
            out = out[:, :vocab]
    d = LogprobDims(N, vocab, ld, 0, dtype_code(logits.dtype), _id_bytes(targets))
    _run(load().lstm_logprob_bwd(ctypes.byref(d), _at(logits), _at(targets), st.inv_temp,
                                 _at(st._buf), _at(st.entropy), _at(dlogp), _at(dentropy),
                                 _at(out), ldd, here), "lstm_logprob_bwd")
    return out


GDR_CHUNK = 64
GDR_STEP_TOKENS = 12


def gdr_dims(T: int, B: int, Hk: int, Hv: int, K: int, V: int, dtype, ldq: int = 0, ldk: int = 0,
             ldv: int = 0) -> GdrDims:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return GdrDims(int(T), int(B), int(Hk), int(Hv), int(K), int(V), code, int(ldq), int(ldk),
                   int(ldv))


def gdr_fwd_workspace_size(d: GdrDims, save: bool = False) -> int:
    return int(load().lstm_gdr_fwd_workspace_size(ctypes.byref(d), int(save)))


def gdr_bwd_workspace_size(d: GdrDims) -> int:
    return int(load().lstm_gdr_bwd_workspace_size(ctypes.byref(d)))


def _sizes_of(d: GdrDims) -> tuple:
    return d.T, d.B, d.Hk, d.Hv, d.K, d.V, d.dtype


class GdrState:
    """Outputs of one gdr_forward() call; states, deltas and ws (save=True; ws
    only where the call allocated it) are kept for the backward."""

    def __init__(self, d: GdrDims, q, save, sT=None, scale=None, lengths=None, made_on=None):
        f = torch.float32
        T, B, H, K, V = d.T, d.B, d.Hv, d.K, d.V
        self.dims, self.scale, self.lengths, self.made_on = d, scale, lengths, made_on
        self.o = q.new_empty(T, B, H, V)
        self.sT = q.new_empty(B, H, K, V, dtype=f) if sT is None else sT
        self.states = self.deltas = self.ws = None
        if save:
            self.states = q.new_empty((-(-T // GDR_CHUNK), B, H, K, V), dtype=f)
            self.deltas = q.new_empty((T, B, H, V), dtype=f)


class GdrGrads:
    def __init__(self, d: GdrDims, cd, device):
        f = dict(dtype=torch.float32, device=device)
        self.dq = torch.empty((d.T, d.B, d.Hk, d.K), dtype=cd, device=device)
        self.dk = torch.empty((d.T, d.B, d.Hk, d.K), dtype=cd, device=device)
        self.dv = torch.empty((d.T, d.B, d.Hv, d.V), dtype=cd, device=device)
        self.dg = torch.empty((d.T, d.B, d.Hv), **f)
        self.dbeta = torch.empty((d.T, d.B, d.Hv), **f)
        self.ds0 = torch.empty((d.B, d.Hv, d.K, d.V), **f)


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the tokens (rows t * B + n) of a [T, B, H, D] tensor
    whose heads are dense: a slice of a wider [T, B, ...] tensor qualifies."""
    T, B, H, D = t.shape
    dense = H * D
    if t.is_contiguous():
        return dense
    _need((D <= 1 or t.stride(3) == 1) and (H <= 1 or t.stride(2) == D),
          f"{name}: heads must be dense")
    ld = t.stride(1) if B > 1 else t.stride(0) if T > 1 else dense
    _need(T <= 1 or B <= 1 or t.stride(0) == B * ld, f"{name}: tokens must have one stride")
    _need(ld >= dense, f"{name}: tokens overlap")
    return ld


def _gdr_call(q, k, v, g, beta, lengths, scale, **dense):
    """(dims, options) of one call, its arguments checked; `dense` are its
    other contiguous tensors."""
    _need(q.dim() == 4 and v.dim() == 4, "q, k [T, B, Hk, K] and v [T, B, Hv, V]")
    T, B, Hk, K = shape = q.shape
    _, _, Hv, V = v.shape
    dt, f = q.dtype, torch.float32
    _sizes(T, B, Hk, Hv, K, V)
    _on(q, k=k, v=v)
    _flat(q, g=g, beta=beta, lengths=lengths, **dense)
    _shaped(k, "k", shape, dt)
    _shaped(v, "v", (T, B, Hv, V), dt)
    _shaped(g, "g", (T, B, Hv), f)
    _shaped(beta, "beta", (T, B, Hv), f)
    _shaped(lengths, "lengths", (B,), torch.int32)
    d = GdrDims(T, B, Hk, Hv, K, V, dtype_code(dt), _token_stride(q, "q"), _token_stride(k, "k"),
                _token_stride(v, "v"))
    return d, GdrOptions(_at(lengths), max(K, 1) ** -0.5 if scale is None else float(scale))


def gdr_forward(q, k, v, g, beta, s0=None, lengths=None, scale=None, save: bool = False, sT=None,
                ws=None, stream=None) -> GdrState:
    """lstm_gdr_fwd: the gated delta rule on q, k [T,B,Hk,K] and v [T,B,Hv,V]
    (one compute dtype; slices of one projection will do), log decay g and
    beta [T,B,Hv] float32, state s0 [B,Hv,K,V] float32.  lengths [B] int32 marks
    padding; scale defaults to K**-0.5.  save keeps what gdr_backward needs;
    sT gives the final state's tensor (s0 itself for a state kept in place).
    A ws of the caller's is free again after the call; the backward then makes
    the operand tiles of the chunks once more."""
    d, opt = _gdr_call(q, k, v, g, beta, lengths, scale, s0=s0, sT=sT, ws=ws)
    state = (d.B, d.Hv, d.K, d.V)
    _shaped(s0, "s0", state, torch.float32)
    _shaped(sT, "sT", state, torch.float32)
    if _elsewhere(q, stream):
        with _there(q, stream, k, v, g, beta, s0, lengths, sT, ws):
            return gdr_forward(q, k, v, g, beta, s0, lengths, scale, save, sT, ws)
    here = _here(q)
    st = GdrState(d, q, save, sT, opt.scale, lengths, here)
    if ws is None and (save or d.T > GDR_STEP_TOKENS):
        ws = _workspace(q, gdr_fwd_workspace_size(d, save))
        if save:
            st.ws = ws
    _run(load().lstm_gdr_fwd(ctypes.byref(d), ctypes.byref(opt), _at(q), _at(k), _at(v), _at(g),
                             _at(beta), _at(s0), _at(st.o), _at(st.sT), _at(st.states),
                             _at(st.deltas), _at(ws), _ws_bytes(ws) if ws is not None else 0,
                             here), "lstm_gdr_fwd")
    return st


def _same_lengths(kept, given, T: int) -> None:
    """The backward's lengths (clamped to 0 .. T) are the forward's."""
    if kept is not None and given is not None and kept.data_ptr() != given.data_ptr():
        _need(not torch.cuda.is_current_stream_capturing(),
              "a backward inside a graph takes the forward's own lengths tensor")
        _need(torch.equal(kept.clamp(0, T), given.clamp(0, T)), "lengths differ from the forward's")
    _need((kept is None) == (given is None), "lengths differ from the forward's")


def gdr_backward(st: GdrState, q, k, v, g, beta, dout=None, dsT=None, lengths=None, scale=None,
                 ws=None, stream=None) -> GdrGrads:
    """lstm_gdr_bwd on the saved state of gdr_forward(..., save=True), with
    the forward's arguments: dout [T,B,Hv,V] (compute dtype), dsT float32.
    (lengths in another tensor than the forward's are compared with those on
    the host, which waits for the device and is refused inside a graph.)"""
    _need(st.states is not None, "the forward kept nothing: call gdr_forward(..., save=True)")
    d, opt = _gdr_call(q, k, v, g, beta, lengths, scale, dout=dout, dsT=dsT, ws=ws, states=st.states)
    _shaped(dout, "dout", (d.T, d.B, d.Hv, d.V), q.dtype)
    _shaped(dsT, "dsT", (d.B, d.Hv, d.K, d.V), torch.float32)
    _need(_sizes_of(d) == _sizes_of(st.dims), "the state belongs to a forward of other sizes")
    _need(opt.scale == st.scale, f"scale {opt.scale} differs from the forward's {st.scale}")
    if _elsewhere(q, stream):
        with _there(q, stream, k, v, g, beta, dout, dsT, lengths, ws):
            return gdr_backward(st, q, k, v, g, beta, dout, dsT, lengths, scale, ws)
    _same_lengths(st.lengths, lengths, d.T)
    here = _here(q)
    if here != st.made_on:
        _used_here(st.states, st.deltas, st.ws)
    gr = GdrGrads(d, q.dtype, q.device)
    if ws is None:
        ws = _workspace(q, gdr_bwd_workspace_size(d))
    _run(load().lstm_gdr_bwd(ctypes.byref(d), ctypes.byref(opt), _at(dout), _at(dsT), _at(q),
                             _at(k), _at(v), _at(g), _at(beta), _at(st.states), _at(st.deltas),
                             _at(gr.dq), _at(gr.dk), _at(gr.dv), _at(gr.dg), _at(gr.dbeta),
                             _at(gr.ds0), _at(st.ws), _at(ws), _ws_bytes(ws), here),
         "lstm_gdr_bwd")
    return gr
