"""Thin ctypes binding over the C ABI declared in include/la.h.

Argument marshalling only: every step of the computation runs in the CUDA library.  PyTorch supplies
device memory and the current stream.  If the compiled library is missing, ``load_library`` raises;
there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
import threading

LA_F32 = 0
LA_BF16 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libla_gb300.so"
_lock = threading.Lock()
_lib = None

_STATUS = {0: "LA_OK", 1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED", 3: "LA_ERR_WORKSPACE", 4: "LA_ERR_CUDA",
           5: "LA_ERR_TIMEOUT", 6: "LA_ERR_BOUNDS", 7: "LA_ERR_STATE"}


class LAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {la_status_string(status)} ({status})")


def library_path() -> str:
    return os.path.join(_HERE, LIB_NAME)


def load_library():
    """Load the compiled CUDA library (built by ``bwd_la_fwd_gb300.build``); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing: run `python -m bwd_la_fwd_gb300.build` "
                               "(or __graft_entry__.build()); there is no CPU fallback")
        _lib = open_library(path)
        return _lib


def open_library(path: str):
    """A ctypes handle on a build of the library at `path`, with every entry point's C signature set
    (load_library() opens the product build with it; the tests also open the index-checked build)."""
    lib = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.la_version.argtypes = []
    lib.la_version.restype = i
    lib.la_launch_count.argtypes = []
    lib.la_launch_count.restype = ctypes.c_ulonglong
    lib.la_status_string.argtypes = [i]
    lib.la_status_string.restype = ctypes.c_char_p
    lib.la_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.la_workspace_bytes.restype = sz
    lib.la_forward.argtypes = [vp, vp, vp, i, vp, vp, i, i, i, i, i, vp, sz, vp]
    lib.la_forward.restype = i
    lib.la_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, sz, vp]
    lib.la_backward.restype = i
    lib.la_backward_with_forward_state.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, sz, vp]
    lib.la_backward_with_forward_state.restype = i
    lp = ctypes.POINTER(ctypes.c_longlong)
    lib.la_forward_strided.argtypes = [vp, vp, vp, i, vp, vp, i, i, i, i, i, lp, vp, sz, vp]
    lib.la_forward_strided.restype = i
    lib.la_backward_strided.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, lp, i, vp, sz, vp]
    lib.la_backward_strided.restype = i
    lib.la_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, vp]
    lib.la_decode_step.restype = i
    lib.la_state_append.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.la_state_append.restype = i
    lib.la_decode_step_grouped.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, lp, vp]
    lib.la_decode_step_grouped.restype = i
    lib.la_prompt_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.la_prompt_workspace_bytes.restype = sz
    lib.la_prompt.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, lp, vp, sz, vp]
    lib.la_prompt.restype = i
    up, dbl, ll = ctypes.POINTER(ctypes.c_ulonglong), ctypes.c_double, ctypes.c_longlong
    lib.la_rotary_frequencies.argtypes = [i, dbl, i, dbl, dbl, dbl, dbl, up]
    lib.la_rotary_frequencies.restype = i
    for f in (lib.la_rotary, lib.la_rotary_backward):
        f.argtypes = [vp, vp, vp, vp, up, vp, ll, ll, i, ctypes.c_float, i, i, i, i, i, i, i, lp, vp]
        f.restype = i
    lib.la_gated_scan.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, lp, vp]
    lib.la_gated_scan.restype = i
    lib.la_gated_scan_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, lp, vp]
    lib.la_gated_scan_backward.restype = i
    lib.la_gated_scan_step.argtypes = [vp, vp, vp, vp, i, i, i, i, lp, vp]
    lib.la_gated_scan_step.restype = i
    lib.la_get_status.argtypes = [vp, vp]
    lib.la_get_status.restype = i
    lib.la_forward_noalloc.argtypes = [vp, vp, vp, i, vp, vp, i, i, i, i, i, vp]
    lib.la_forward_noalloc.restype = i
    lib.la_noalloc_get_status.argtypes = [vp]
    lib.la_noalloc_get_status.restype = i
    return lib


def la_status_string(status: int) -> str:
    if _lib is not None:
        return _lib.la_status_string(int(status)).decode()
    return _STATUS.get(int(status), "LA_UNKNOWN_STATUS")


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return LA_BF16
    if t.dtype == torch.float32:
        return LA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _shape(Q):
    if Q.dim() != 4:
        raise ValueError(f"expected a [B, H, N, D] tensor, got shape {tuple(Q.shape)}")
    return tuple(int(s) for s in Q.shape)


def _check_like(Q, *others):
    for t in (Q, *others):
        if t is None:
            continue
        if t.shape != Q.shape or t.dtype != Q.dtype or t.device != Q.device:
            raise ValueError("all [B,H,N,D] tensors must share shape, dtype and device")
        if t.stride(-1) != 1:
            raise ValueError("the D elements of each row must be contiguous (stride(-1) == 1)")


def _strides(*ts):
    """(batch, head, row) element strides of each [B,H,N,D] view, as the strided entry points take them."""
    vals = [int(x) for t in ts for x in t.stride()[:3]]
    return (ctypes.c_longlong * len(vals))(*vals)


def la_launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(load_library().la_launch_count())


def la_workspace_bytes(B: int, H: int, N: int, D: int, causal: bool, dtype: int, backward: bool) -> int:
    return int(load_library().la_workspace_bytes(B, H, N, D, int(bool(causal)), int(dtype), int(bool(backward))))


def new_workspace(B: int, H: int, N: int, D: int, causal: bool, dtype: int, backward: bool, device="cuda"):
    """Zero-filled device workspace of the size the library asks for (torch owns it)."""
    import torch
    n = la_workspace_bytes(B, H, N, D, causal, dtype, backward)
    if n == 0:
        raise LAError(1, "la_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def la_forward(Q, K, V, causal: bool, O=None, normaliser=None, workspace=None, stream=None):
    """O, g = la_forward(Q, K, V, causal): normalised linear attention forward on [B,H,N,D] tensors.

    The tensors may be strided views (a [B,N,H,D] tensor permuted to [B,H,N,D], a slice of a fused QKV
    projection) as long as each row's D elements are contiguous; they go to the library as they are."""
    import torch
    B, H, N, D = _shape(Q)
    _check_like(Q, K, V, O)
    dt = _dtype_code(Q)
    if O is None:
        O = torch.empty_like(Q)
    if normaliser is None:
        normaliser = torch.empty((B, H, N), dtype=torch.float32, device=Q.device)
    if workspace is None:
        workspace = new_workspace(B, H, N, D, causal, dt, False, Q.device)
    st = load_library().la_forward_strided(_ptr(Q), _ptr(K), _ptr(V), int(bool(causal)), _ptr(O), _ptr(normaliser),
                                           B, H, N, D, dt, _strides(Q, K, V, O), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != 0:
        raise LAError(st, "la_forward")
    return O, normaliser


def la_backward(Q, K, V, O, dO, causal: bool, dQ=None, dK=None, dV=None, workspace=None, stream=None,
                reuse_forward_state: bool = False):
    """dQ, dK, dV = la_backward(Q, K, V, O, dO, causal): gradients of sum(dO * O).

    With ``reuse_forward_state`` the call is la_backward_with_forward_state: it takes the per-piece state
    sums that the last la_forward on ``workspace`` (same K, V, shape) left there instead of recomputing
    them; the workspace must then be given (and sized for the backward at that forward)."""
    import torch
    B, H, N, D = _shape(Q)
    _check_like(Q, K, V, O, dO, dQ, dK, dV)
    dt = _dtype_code(Q)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(Q) if dK is None else dK
    dV = torch.empty_like(Q) if dV is None else dV
    if workspace is None:
        if reuse_forward_state:
            raise ValueError("reuse_forward_state needs the workspace the forward ran with")
        workspace = new_workspace(B, H, N, D, causal, dt, True, Q.device)
    st = load_library().la_backward_strided(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV),
                                            int(bool(causal)), B, H, N, D, dt, _strides(Q, K, V, O, dO, dQ, dK, dV),
                                            int(bool(reuse_forward_state)), _ptr(workspace),
                                            workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != 0:
        raise LAError(st, "la_backward_with_forward_state" if reuse_forward_state else "la_backward")
    return dQ, dK, dV


def la_get_status(workspace, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status recorded in the workspace."""
    return int(load_library().la_get_status(_ptr(workspace), _stream_ptr(stream)))


def la_forward_noalloc(Q, K, V, causal: bool, O=None, normaliser=None, stream=None):
    """The forward without a workspace argument: the library's fixed scratch array on the current device
    serves instead (for callers that cannot allocate device memory).  Returns (O, normaliser)."""
    import torch
    B, H, N, D = _shape(Q)
    _check_like(Q, K, V)
    if O is None:
        O = torch.empty_like(Q)
    if normaliser is None:
        normaliser = torch.empty((B, H, N), device=Q.device, dtype=torch.float32)
    st = load_library().la_forward_noalloc(_ptr(Q), _ptr(K), _ptr(V), int(bool(causal)), _ptr(O), _ptr(normaliser),
                                           B, H, N, D, _dtype_code(Q), _stream_ptr(stream))
    if st != 0:
        raise LAError(st, "la_forward_noalloc")
    return O, normaliser


def la_noalloc_get_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status of the fixed scratch array."""
    return int(load_library().la_noalloc_get_status(_stream_ptr(stream)))


class DecodeState:
    """The carried state of the recurrent (decode) form, per (b, h): S [B,H,D,D], z [B,H,D], a [B,H,D] of
    the accumulator type (float32 for bf16 tokens, float64 for float32 tokens) and the count n (int32
    [B,H]).  Zero-filled is the empty state; the library updates the tensors in place.

    For grouped heads H is the number of key/value heads.  ``tensors`` = (S, z, a, n) takes the caller's
    tensors (parts of a larger cache, say) instead of new ones."""

    def __init__(self, B: int, H: int, D: int, token_dtype, device="cuda", tensors=None):
        import torch
        acc = torch.float32 if token_dtype == torch.bfloat16 else torch.float64
        if token_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"unsupported dtype {token_dtype}: use torch.bfloat16 or torch.float32")
        self.B, self.H, self.D, self.token_dtype = B, H, D, token_dtype
        if tensors is not None:
            for t, shape, dt in zip(tensors, ((B, H, D, D), (B, H, D), (B, H, D), (B, H)), (acc, acc, acc, torch.int32)):
                if tuple(t.shape) != shape or t.dtype != dt or not t.is_contiguous() or t.device != tensors[0].device:
                    raise ValueError(f"expected a contiguous {dt} tensor of shape {shape} on one device")
            self.S, self.z, self.a, self.n = tensors
            return
        self.S = torch.zeros((B, H, D, D), dtype=acc, device=device)
        self.z = torch.zeros((B, H, D), dtype=acc, device=device)
        self.a = torch.zeros((B, H, D), dtype=acc, device=device)
        self.n = torch.zeros((B, H), dtype=torch.int32, device=device)

    def _args(self):
        return _ptr(self.S), _ptr(self.z), _ptr(self.a), _ptr(self.n)


def la_decode_step(state: DecodeState, q, k, v, o=None, normaliser=None, stream=None):
    """o, g = la_decode_step(state, q, k, v): append one token per (b, h) ([B,H,D] tensors) to ``state``
    and return its output and normaliser (row n - 1 of the causal forward over the tokens taken so far)."""
    import torch
    if q.dim() != 3 or tuple(q.shape) != (state.B, state.H, state.D):
        raise ValueError(f"expected [B, H, D] = {(state.B, state.H, state.D)} tokens, got {tuple(q.shape)}")
    for t in (k, v, o):
        if t is not None and (t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous()):
            raise ValueError("q, k, v, o must share shape and dtype and be contiguous")
    if q.dtype != state.token_dtype:
        raise ValueError("token dtype does not match the state")
    o = torch.empty_like(q) if o is None else o
    if normaliser is None:
        normaliser = torch.empty((state.B, state.H), dtype=torch.float32, device=q.device)
    st = load_library().la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(normaliser), *state._args(),
                                       state.B, state.H, state.D, _dtype_code(q), _stream_ptr(stream))
    if st != 0:
        raise LAError(st, "la_decode_step")
    return o, normaliser


def la_state_append(state: DecodeState, K, V, stream=None):
    """Append N tokens per (b, h) ([B,H,N,D] tensors) to ``state``: S += K^T V, z += sum k, a += sum v,
    n += N."""
    B, H, N, D = _shape(K)
    _check_like(K, V)
    if (B, H, D) != (state.B, state.H, state.D) or K.dtype != state.token_dtype:
        raise ValueError("K, V do not match the state's B, H, D and token dtype")
    st = load_library().la_state_append(_ptr(K), _ptr(V), *state._args(), B, H, N, D, _dtype_code(K),
                                        _stream_ptr(stream))
    if st != 0:
        raise LAError(st, "la_state_append")
    return state


class _on:
    """Makes a stream and its device the current ones for a call: new tensors belong to that stream, and the library
    launches on that device."""

    __slots__ = ("_ctx",)

    def __init__(self, ctx):
        self._ctx = ctx

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


_HERE_ALREADY = _on(None)


def _place(stream, first, *ts):
    """(context, stream pointer) of a call on these tensors, all of one CUDA device: on `stream`, or on the current
    stream of their device."""
    import torch
    dev = first.device
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on one device, got {dev} and {t.device}")
    index = dev.index
    if index is None or dev.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got {dev}")
    if stream is None:
        here = torch._C._cuda_getDevice() == index
        return _HERE_ALREADY if here else _on(torch.cuda.device(dev)), torch._C._cuda_getCurrentRawStream(index)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return _on(torch.cuda.stream(stream)), stream.cuda_stream


_ARRAYS = {n: ctypes.c_longlong * n for n in (3, 6, 8, 12)}


def _rows(t):
    """A tensor's strides; its last dimension has to be contiguous."""
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1:
        raise ValueError("the last dimension must be contiguous (stride(-1) == 1)")
    return s


def _expect(t, shape, dtype, what):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")


def la_decode_step_grouped(state: DecodeState, q, k, v, o=None, normaliser=None, stream=None):
    """o = la_decode_step_grouped(state, q, k, v): one token for grouped heads, q [B,Hq,D], k and v [B,Hkv,D] with
    Hkv = state.H and Hq a multiple of it.  The tensors may be strided views (slices of a fused projection) with
    contiguous D; `normaliser`, if given, is a float32 [B,Hq] tensor that receives g."""
    import torch
    B, H, D = state.B, state.H, state.D
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or shape[0] != B or shape[2] != D or H < 1 or shape[1] % H != 0 or shape[1] < H:
        raise ValueError(f"expected [B, r Hkv, D] queries for B, Hkv, D = {(B, H, D)}, got {tuple(shape)}")
    Hq = shape[1]
    if k.shape != (B, H, D) or v.shape != (B, H, D) or (o is not None and o.shape != shape):
        raise ValueError(f"expected k, v of shape {(B, H, D)} and o like q")
    if dtype != state.token_dtype or k.dtype != dtype or v.dtype != dtype or (o is not None and o.dtype != dtype):
        raise ValueError("token dtype does not match the state")
    if normaliser is not None:
        _expect(normaliser, (B, Hq), torch.float32, "normaliser")
    sq, sk, sv = _rows(q), _rows(k), _rows(v)
    so = (Hq * D, D) if o is None else _rows(o)
    on, sp = _place(stream, q, k, v, o, normaliser, state.S, state.z, state.a, state.n)
    with on:
        if o is None:
            o = torch.empty(shape, dtype=dtype, device=q.device)
        st = load_library().la_decode_step_grouped(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), 0 if normaliser is None else normaliser.data_ptr(),
            state.S.data_ptr(), state.z.data_ptr(), state.a.data_ptr(), state.n.data_ptr(), B, Hq, H, D, _dtype_code(q),
            _ARRAYS[8](sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1]), sp)
    if st != 0:
        raise LAError(st, "la_decode_step_grouped")
    return o


def la_prompt_workspace_bytes(T: int, nseq: int, Hq: int, Hkv: int, D: int, dtype: int) -> int:
    return int(load_library().la_prompt_workspace_bytes(T, nseq, Hq, Hkv, D, int(dtype)))


def new_prompt_workspace(T: int, nseq: int, Hq: int, Hkv: int, D: int, dtype: int, device="cuda"):
    """Zero-filled device workspace of the size la_prompt asks for."""
    import torch
    n = la_prompt_workspace_bytes(T, nseq, Hq, Hkv, D, dtype)
    if n == 0:
        raise LAError(1, "la_prompt_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def la_prompt(Q, K, V, seq_offsets, state=None, resume: bool = False, O=None, workspace=None, stream=None):
    """O = la_prompt(Q, K, V, seq_offsets, state): the causal forward over packed prompts with grouped heads.

    Q [T,Hq,D], K and V [T,Hkv,D] (strided views with contiguous D are taken as they are); sequence i has rows
    seq_offsets[i] ... seq_offsets[i+1] - 1 (int32 on the device).  ``state``, a DecodeState(nseq, Hkv, D), receives
    each sequence's state, or with ``resume`` continues from it.  Rows outside every sequence keep what O holds (a new
    O is zero there).  Offsets that are not in order within [0, T] compute nothing, and la_get_status(workspace) tells so:
    a caller that does not know them to be in order passes a ``workspace`` (new_prompt_workspace; one for the largest T and
    nseq serves smaller calls too).  One made for a single call, and zeroed for it, is gone with its status."""
    import torch
    if Q.dim() != 3 or K.dim() != 3 or seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
        raise ValueError("expected [T, H, D] tensors and [nseq + 1] offsets")
    T, Hq, D = Q.shape
    Hkv, nseq = K.shape[1], seq_offsets.shape[0] - 1
    if K.shape[0] != T or K.shape[2] != D or V.shape != K.shape or (O is not None and O.shape != Q.shape):
        raise ValueError(f"Q {tuple(Q.shape)}, K {tuple(K.shape)}, V {tuple(V.shape)} do not match")
    if Hkv < 1 or Hq < Hkv or Hq % Hkv != 0:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} key/value heads")
    for t in (K, V, O):
        if t is not None and t.dtype != Q.dtype:
            raise ValueError("Q, K, V, O must share their dtype")
    _expect(seq_offsets, (nseq + 1,), torch.int32, "seq_offsets")
    dt = _dtype_code(Q)
    if state is not None and ((state.B, state.H, state.D) != (nseq, Hkv, D) or state.token_dtype != Q.dtype):
        raise ValueError(f"the state is not one of nseq, Hkv, D = {(nseq, Hkv, D)} and {Q.dtype}")
    if resume and state is None:
        raise ValueError("resume needs a state")
    parts = (state.S, state.z, state.a, state.n) if state is not None else (None,) * 4
    on, sp = _place(stream, Q, K, V, O, seq_offsets, workspace, *parts)
    with on:
        if O is None:
            O = torch.zeros((T, Hq, D), dtype=Q.dtype, device=Q.device)
        strides = [s for t in (Q, K, V, O) for s in _rows(t)[1::-1]]  # (head, row)
        if workspace is None:
            workspace = new_prompt_workspace(T, nseq, Hq, Hkv, D, dt, Q.device)
        st = load_library().la_prompt(
            Q.data_ptr(), K.data_ptr(), V.data_ptr(), seq_offsets.data_ptr(), O.data_ptr(), *map(_ptr, parts),
            int(bool(resume)), T, nseq, Hq, Hkv, D, dt,
            _ARRAYS[8](*strides), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), sp)
    if st != 0:
        raise LAError(st, "la_prompt")
    return O


class RotaryFrequencies:
    """The rotation of each channel pair per position, in units of 2^-64 turns (``values``, a host array that the
    library reads during each call), for heads of which ``rotary_dim`` channels are rotated."""

    def __init__(self, rotary_dim: int, values):
        self.rotary_dim = int(rotary_dim)
        self.values = (ctypes.c_ulonglong * (self.rotary_dim // 2))(*values)


_ROTARY_SCALING = {"none": 0, "linear": 1, "by_turns": 2}


def la_rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                          original_length: float = 0.0, low_turns: float = 1.0, high_turns: float = 32.0):
    """RotaryFrequencies for base^(-2 i / rotary_dim) radians per position: as they are ("none"), divided by `factor`
    ("linear"), or divided by it only for the pairs of few turns over `original_length` positions ("by_turns")."""
    if scaling not in _ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY_SCALING)}")
    out = (ctypes.c_ulonglong * max(1, int(rotary_dim) // 2))()
    st = load_library().la_rotary_frequencies(int(rotary_dim), base, _ROTARY_SCALING[scaling], factor, original_length,
                                              low_turns, high_turns, out)
    if st != 0:
        raise LAError(st, "la_rotary_frequencies")
    return RotaryFrequencies(rotary_dim, out)


def _rotary(name, Q, K, freqs, positions, first_position, interleaved, magnitude, Q_out, K_out, stream):
    import torch
    shape, dtype, Hk = Q.shape, Q.dtype, 0
    if len(shape) != 4:
        raise ValueError(f"expected a [B, H, N, D] tensor, got shape {tuple(shape)}")
    B, Hq, N, D = shape
    if K is not None:
        ks = K.shape
        if len(ks) != 4 or ks[0] != B or ks[2] != N or ks[3] != D or K.dtype != dtype:
            raise ValueError("Q and K must be [B, H, N, D] tensors that share B, N, D and dtype")
        Hk = ks[1]
    elif K_out is not None:
        raise ValueError("K_out without K")
    for out, like in ((Q_out, Q), (K_out, K)):
        if out is not None and (out.shape != like.shape or out.dtype != dtype):
            raise ValueError("the outputs must share their inputs' shape and dtype")
    dt, ps = _dtype_code(Q), 0
    if positions is not None:
        ext = positions.shape
        if positions.dtype != torch.int32 or (ext != (B, N) and ext != (N,)) or (N > 1 and positions.stride(-1) != 1):
            raise ValueError(f"positions: expected int32 [N] or [B, N] with contiguous rows, got {positions.dtype} "
                             f"{tuple(ext)}")
        # a batch of one is stepped by nothing, whatever its stride
        ps = positions.stride(0) if len(ext) == 2 and B > 1 else 0
        if ps and ps < N:
            raise ValueError("positions of the batch entries overlap")
    sq = _rows(Q)
    sk = _rows(K) if Hk else (0, 0, 0)
    sqo = (Hq * N * D, N * D, D) if Q_out is None else _rows(Q_out)
    sko = (Hk * N * D, N * D, D) if K_out is None else _rows(K_out)
    on, sp = _place(stream, Q, K, Q_out, K_out, positions)
    with on:
        if Q_out is None:
            Q_out = torch.empty(shape, dtype=dtype, device=Q.device)
        if K is not None and K_out is None:
            K_out = torch.empty(ks, dtype=dtype, device=Q.device)
        st = getattr(load_library(), name)(
            Q.data_ptr(), K.data_ptr() if Hk else 0, Q_out.data_ptr(), K_out.data_ptr() if Hk else 0, freqs.values,
            0 if positions is None else positions.data_ptr(), ps, first_position, 1 if interleaved else 0, magnitude, B, Hq,
            Hk, N, D, freqs.rotary_dim, dt,
            _ARRAYS[12](sq[0], sq[1], sq[2], sk[0], sk[1], sk[2], sqo[0], sqo[1], sqo[2], sko[0], sko[1], sko[2]), sp)
    if st != 0:
        raise LAError(st, name)
    return Q_out, K_out


def la_rotary(Q, K, freqs: RotaryFrequencies, positions=None, first_position: int = 0, interleaved: bool = False,
              magnitude: float = 1.0, Q_out=None, K_out=None, stream=None):
    """Q', K' = la_rotary(Q, K, freqs): positions rotated into Q [B,Hq,N,D] and K [B,Hk,N,D] (or None), in one launch.

    ``positions`` is an int32 [B,N] or [N] device tensor; without it row i has position first_position + i.  Views
    with contiguous D are taken as they are; Q_out = Q and K_out = K rotate in place."""
    return _rotary("la_rotary", Q, K, freqs, positions, first_position, interleaved, magnitude, Q_out, K_out, stream)


def la_rotary_backward(dQ, dK, freqs: RotaryFrequencies, positions=None, first_position: int = 0,
                       interleaved: bool = False, magnitude: float = 1.0, dQ_out=None, dK_out=None, stream=None):
    """The gradients of la_rotary's inputs from those of its outputs (the other arguments as given to it)."""
    return _rotary("la_rotary_backward", dQ, dK, freqs, positions, first_position, interleaved, magnitude, dQ_out,
                   dK_out, stream)


_GATES = {"log": 0, "sigmoid": 1}


def _gate_code(gate) -> int:
    if gate not in _GATES:
        raise ValueError(f"gate must be one of {sorted(_GATES)}")
    return _GATES[gate]


def _scan_operands(dims, first, *others):
    """The operands' row strides ((batch, row) each); None, an output that the call makes, is contiguous."""
    shape, dtype = first.shape, first.dtype
    if len(shape) != dims:
        raise ValueError(f"expected a {'[B, N, C]' if dims == 3 else '[B, C]'} tensor, got shape {tuple(shape)}")
    strides = list(_rows(first)[:-1])
    dense = (shape[1] * shape[2], shape[2]) if dims == 3 else (shape[1],)
    for t in others:
        if t is None:
            strides += dense
            continue
        if t.shape != shape or t.dtype != dtype:
            raise ValueError("the tensors must share shape and dtype")
        strides += _rows(t)[:-1]
    return strides


def la_gated_scan(X, W, gate: str, h0=None, H=None, h_last=None, stream=None):
    """H, h_last = la_gated_scan(X, W, gate): h_t = a_t h_{t-1} + b_t x_t along dimension 1 of [B,N,C] tensors, per
    channel, with a = e^w, b = 1 (gate "log") or a = sigmoid(w), b = 1 - a (gate "sigmoid").  h0 and h_last are float32
    [B,C]: the value before the first row (None: 0) and after the last."""
    import torch
    strides = _scan_operands(3, X, W, H)
    B, N, C = X.shape
    code, dt = _gate_code(gate), _dtype_code(X)
    for t, what in ((h0, "h0"), (h_last, "h_last")):
        if t is not None:
            _expect(t, (B, C), torch.float32, what)
    on, sp = _place(stream, X, W, h0, H, h_last)
    with on:
        if H is None:
            H = torch.empty((B, N, C), dtype=X.dtype, device=X.device)
        if h_last is None:
            h_last = torch.empty((B, C), dtype=torch.float32, device=X.device)
        st = load_library().la_gated_scan(X.data_ptr(), W.data_ptr(), _ptr(h0), H.data_ptr(), h_last.data_ptr(), B, N, C,
                                          code, dt, _ARRAYS[6](*strides),
                                          sp)
    if st != 0:
        raise LAError(st, "la_gated_scan")
    return H, h_last


def la_gated_scan_backward(X, W, H, dH, gate: str, h0=None, dh_last=None, dX=None, dW=None, dh0=None, stream=None):
    """dX, dW, dh0 = la_gated_scan_backward(X, W, H, dH, gate): gradients of sum(dH * H) + sum(dh_last * h_last), H and
    h0 as the forward had them."""
    import torch
    strides = _scan_operands(3, X, W, H, dH, dX, dW)
    B, N, C = X.shape
    code, dt = _gate_code(gate), _dtype_code(X)
    for t, what in ((h0, "h0"), (dh_last, "dh_last"), (dh0, "dh0")):
        if t is not None:
            _expect(t, (B, C), torch.float32, what)
    on, sp = _place(stream, X, W, H, dH, h0, dh_last, dX, dW, dh0)
    with on:
        dX = torch.empty((B, N, C), dtype=X.dtype, device=X.device) if dX is None else dX
        dW = torch.empty((B, N, C), dtype=X.dtype, device=X.device) if dW is None else dW
        dh0 = torch.empty((B, C), dtype=torch.float32, device=X.device) if dh0 is None else dh0
        st = load_library().la_gated_scan_backward(
            X.data_ptr(), W.data_ptr(), H.data_ptr(), dH.data_ptr(), _ptr(h0), _ptr(dh_last), dX.data_ptr(),
            dW.data_ptr(), dh0.data_ptr(), B, N, C, code, dt,
            _ARRAYS[12](*strides), sp)
    if st != 0:
        raise LAError(st, "la_gated_scan_backward")
    return dX, dW, dh0


def la_gated_scan_step(state, x, w, gate: str, h=None, stream=None):
    """h = la_gated_scan_step(state, x, w, gate): one row of the recurrence for [B,C] tensors; ``state``, float32 [B,C],
    is advanced in place."""
    import torch
    strides = _scan_operands(2, x, w, h)
    B, C = x.shape
    code, dt = _gate_code(gate), _dtype_code(x)
    _expect(state, (B, C), torch.float32, "state")
    on, sp = _place(stream, x, w, h, state)
    with on:
        if h is None:
            h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        st = load_library().la_gated_scan_step(x.data_ptr(), w.data_ptr(), h.data_ptr(), state.data_ptr(), B, C, code, dt,
                                               _ARRAYS[3](*strides), sp)
    if st != 0:
        raise LAError(st, "la_gated_scan_step")
    return h
