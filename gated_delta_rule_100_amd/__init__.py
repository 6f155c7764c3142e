"""gated_delta_rule_100_amd -- the gated delta rule on AMD Instinct MI355X.

Python binding of libgdr.so (the C ABI declared in include/gdr.h).  It only
marshals arguments: it takes torch device tensors (torch is used for device
memory and streams), checks their dtype/shape/placement, and passes raw
pointers and sizes to the library.  Every step of the computation runs in the
HIP kernels of libgdr; there is no CPU path.  If the library is not built, or
a tensor is not on the GPU, the call raises.

    S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = S_t q_t,
    alpha_t = exp(g_t), state S of shape dv x dk per (sequence, head).
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "GdrError",
    "GDR_BF16",
    "GDR_FP32",
    "library_path",
    "gdr_decode_step",
    "gdr_decode_mtp",
    "gdr_chunk_prefill",
    "gdr_chunk_prefill_noalloc",
    "gdr_chunk_prefill_workspace_bytes",
    "gdr_state_fixup",
    "gdr_chunk_layout",
    "gdr_max_chunks",
    "gdr_linear_decode",
    "gdr_linear_prefill",
    "gdr_linear_prefill_workspace_bytes",
    "gdr_linear_backward",
    "gdr_linear_backward_workspace_bytes",
    "gdr_block_norm",
    "gdr_block_norm_backward",
    "gdr_block_norm_backward_workspace_bytes",
    "gdr_status_string",
    "gdr_last_error",
]

GDR_BF16 = 0
GDR_FP32 = 1
GDR_DECAY_TOKEN = 0
GDR_DECAY_HEAD = 1
GDR_GATES = {"silu": 0, "sigmoid": 1}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libgdr.so")
_lib = None


class GdrError(RuntimeError):
    """A libgdr call returned a non-OK status."""


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise GdrError(f"{_LIB_PATH} is missing: build it with gated_delta_rule_100_amd/build.py "
                       "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.gdr_decode_step.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
    lib.gdr_decode_mtp.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]
    lib.gdr_decode_step.restype = I
    lib.gdr_decode_mtp.restype = I
    lib.gdr_max_chunks.argtypes = [I, I, I]
    lib.gdr_max_chunks.restype = I
    lib.gdr_chunk_layout.argtypes = [P, I, I, P, P, I, P]
    lib.gdr_chunk_layout.restype = I
    lib.gdr_chunk_prefill_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.gdr_chunk_prefill_workspace_bytes.restype = S
    lib.gdr_chunk_prefill.argtypes = [P, P, P, P, P, P, I, P, P, P, P, P, P,
                                      I, I, I, I, I, I, I, P, S, P]
    lib.gdr_chunk_prefill.restype = I
    lib.gdr_chunk_prefill_noalloc.argtypes = [P, P, P, P, P, P, I, P, P, P, P, P, P,
                                              I, I, I, I, I, I, I, P]
    lib.gdr_chunk_prefill_noalloc.restype = I
    lib.gdr_state_fixup.argtypes = [P, P, P, P, I, P, I, I, I, I, P]
    lib.gdr_state_fixup.restype = I
    L, F = ctypes.c_int64, ctypes.c_float
    lib.gdr_linear_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, L, L, L, F, I, I, I, P]
    lib.gdr_linear_decode.restype = I
    lib.gdr_linear_prefill.argtypes = [P, P, P, P, P, I, P, P, P, I, I, I, I, I, L, L, L, F, I, I,
                                       I, P, S, P]
    lib.gdr_linear_prefill.restype = I
    lib.gdr_linear_prefill_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gdr_linear_prefill_workspace_bytes.restype = S
    lib.gdr_linear_backward.argtypes = [P, P, P, P, P, I, P, P, P, P, P, P, P, P, I, I, I, I, I,
                                        L, L, L, F, I, I, I, P, S, P]
    lib.gdr_linear_backward.restype = I
    lib.gdr_linear_backward_workspace_bytes.argtypes = [I, I, I, I, I, I, I]
    lib.gdr_linear_backward_workspace_bytes.restype = S
    lib.gdr_block_norm.argtypes = [P] * 7 + [L, I, F, F, I, I, I, I, P]
    lib.gdr_block_norm.restype = I
    lib.gdr_block_norm_backward.argtypes = [P] * 12 + [L, I, F, F, I, I, I, I, P, S, P]
    lib.gdr_block_norm_backward.restype = I
    lib.gdr_block_norm_backward_workspace_bytes.argtypes = [L, I]
    lib.gdr_block_norm_backward_workspace_bytes.restype = S
    lib.gdr_status_string.argtypes = [I]
    lib.gdr_status_string.restype = ctypes.c_char_p
    lib.gdr_last_error.argtypes = []
    lib.gdr_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def gdr_status_string(status: int) -> str:
    return _load().gdr_status_string(status).decode()


def gdr_last_error() -> str:
    return _load().gdr_last_error().decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise GdrError(f"{what}: {gdr_status_string(status)}: {gdr_last_error()}")


def _dev_ptr(t, name, dtypes=None, optional=False):
    if t is None:
        if optional:
            return None
        raise GdrError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GdrError(f"{name} must be a torch tensor on the GPU")
    if not t.is_contiguous():
        raise GdrError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise GdrError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


def _code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return GDR_BF16
    if dt == torch.float32:
        return GDR_FP32
    raise GdrError(f"unsupported dtype {dt}")


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_IO = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def gdr_decode_step(q, k, v, g, beta, state, o, stream=None, *, norm=None) -> None:
    """One decode token, state updated in place.  q, k [N, H, dk], v [N, H, dv]
    (bf16 or fp32, one dtype); g, beta [N, H] fp32; state [N, H, dv, dk] fp32;
    o [N, H, dv] bf16 or fp32.  norm: a dict of gdr_block_norm's arguments after
    x (h, y, w_after, gate, ...): the norm and gate behind the heads, of every
    row of o, on the same stream; what it would refuse is refused before
    anything runs."""
    N, H, dk = q.shape
    dv = v.shape[2]
    if k.shape != q.shape or v.shape[:2] != (N, H) or g.shape != (N, H) or beta.shape != (N, H) \
            or state.shape != (N, H, dv, dk) or o.shape != (N, H, dv):
        raise GdrError("gdr_decode_step: inconsistent shapes")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise GdrError("gdr_decode_step: q, k, v must share a dtype")
    dev = _device(q, "q")
    after = _norm_after(o, norm, dev, stream)
    _launch("gdr_decode_step", _load().gdr_decode_step, dev, stream,
            _dev_ptr(q, "q", _IO), _dev_ptr(k, "k", _IO), _dev_ptr(v, "v", _IO),
            _dev_ptr(g, "g", _F32), _dev_ptr(beta, "beta", _F32), _dev_ptr(state, "state", _F32),
            _dev_ptr(o, "o", _IO), N, H, dk, dv, _code(q.dtype), _code(o.dtype))
    after()


def gdr_decode_mtp(q, k, v, g, beta, state_in, state_out, o, inter=None, stream=None, *,
                   norm=None) -> None:
    """T decode tokens per (sequence, head).  q, k [N, T, H, dk], v [N, T, H, dv]
    (bf16 or fp32, one dtype); g, beta [N, T, H] fp32; state_in [N, H, dv, dk]
    fp32; state_out like state_in, the same tensor (in place) or None (no final
    state written); o [N, T, H, dv] bf16 or fp32; inter [N, T, H, dv, dk] fp32
    or None (the state after every token).  norm: as gdr_decode_step's."""
    N, T, H, dk = q.shape
    dv = v.shape[3]
    if k.shape != q.shape or v.shape[:3] != (N, T, H) or g.shape != (N, T, H) \
            or beta.shape != (N, T, H) or state_in.shape != (N, H, dv, dk) \
            or o.shape != (N, T, H, dv) \
            or (state_out is not None and state_out.shape != state_in.shape) \
            or (inter is not None and inter.shape != (N, T, H, dv, dk)):
        raise GdrError("gdr_decode_mtp: inconsistent shapes")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise GdrError("gdr_decode_mtp: q, k, v must share a dtype")
    dev = _device(q, "q")
    after = _norm_after(o, norm, dev, stream)
    _launch("gdr_decode_mtp", _load().gdr_decode_mtp, dev, stream,
            _dev_ptr(q, "q", _IO), _dev_ptr(k, "k", _IO), _dev_ptr(v, "v", _IO),
            _dev_ptr(g, "g", _F32), _dev_ptr(beta, "beta", _F32),
            _dev_ptr(state_in, "state_in", _F32),
            _dev_ptr(state_out, "state_out", _F32, optional=True),
            _dev_ptr(o, "o", _IO), _dev_ptr(inter, "inter", _F32, optional=True), N, T, H, dk, dv,
            _code(q.dtype), _code(o.dtype))
    after()


def gdr_max_chunks(T_total: int, N: int, chunk: int) -> int:
    return int(_load().gdr_max_chunks(T_total, N, chunk))


def gdr_chunk_prefill_workspace_bytes(T_total, N, H, dk, dv, chunk, in_dtype=GDR_BF16) -> int:
    """in_dtype: GDR_BF16 / GDR_FP32 or the torch dtype of q, k, v."""
    if isinstance(in_dtype, torch.dtype):
        in_dtype = _code(in_dtype)
    return int(_load().gdr_chunk_prefill_workspace_bytes(T_total, N, H, dk, dv, chunk, in_dtype))


def gdr_chunk_layout(cu_seqlens, chunk, chunk_offsets, chunk_indices, stream=None) -> None:
    """cu_seqlens [N+1] int32 -> chunk_offsets [N+1] int32, chunk_indices
    [max_chunks, 2] int32 (rows past the real count = (-1, -1))."""
    N = cu_seqlens.shape[0] - 1
    if chunk_offsets.shape != (N + 1,) or chunk_indices.dim() != 2 or chunk_indices.shape[1] != 2:
        raise GdrError("gdr_chunk_layout: inconsistent shapes")
    st = _load().gdr_chunk_layout(
        _dev_ptr(cu_seqlens, "cu_seqlens", _I32), N, chunk,
        _dev_ptr(chunk_offsets, "chunk_offsets", _I32),
        _dev_ptr(chunk_indices, "chunk_indices", _I32), chunk_indices.shape[0], _stream(stream))
    _check(st, "gdr_chunk_layout")


def _prefill_args(q, k, v, g, beta, cu_seqlens, state_in, state_out, o, chunk, L_out, M_out,
                  fixed_out, who):
    """Checks the shapes and dtypes of a prefill call; returns the pointer and
    size arguments shared by gdr_chunk_prefill and gdr_chunk_prefill_noalloc
    (everything up to out_dtype) and (T, N, H, dk, dv)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = cu_seqlens.shape[0] - 1
    if k.shape != q.shape or v.shape[:2] != (T, H) or g.shape != (T, H) or beta.shape != (T, H) \
            or state_out.shape != (N, H, dv, dk) or o.shape != (T, H, dv) \
            or (state_in is not None and state_in.shape != (N, H, dv, dk)):
        raise GdrError(f"{who}: inconsistent shapes")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise GdrError(f"{who}: q, k, v must share a dtype")
    mc = gdr_max_chunks(T, N, chunk)
    for name, t, shape in (("L_out", L_out, (mc, H, dv, dk)), ("M_out", M_out, (mc, H, dk, dk)),
                           ("fixed_out", fixed_out, (mc, H, dv, dk))):
        if t is not None and tuple(t.shape) != shape:
            raise GdrError(f"{who}: {name} must have shape {shape}")
    args = [
        _dev_ptr(q, "q", _IO), _dev_ptr(k, "k", _IO), _dev_ptr(v, "v", _IO),
        _dev_ptr(g, "g", _F32), _dev_ptr(beta, "beta", _F32),
        _dev_ptr(cu_seqlens, "cu_seqlens", _I32), N,
        _dev_ptr(state_in, "state_in", _F32, optional=True),
        _dev_ptr(state_out, "state_out", _F32), _dev_ptr(o, "o", _IO),
        _dev_ptr(L_out, "L_out", _F32, optional=True), _dev_ptr(M_out, "M_out", _F32, optional=True),
        _dev_ptr(fixed_out, "fixed_out", _F32, optional=True),
        T, H, dk, dv, chunk, _code(q.dtype), _code(o.dtype)]
    return args, (T, N, H, dk, dv)


def gdr_chunk_prefill(q, k, v, g, beta, cu_seqlens, state_in, state_out, o, *, chunk=64,
                      L_out=None, M_out=None, fixed_out=None, workspace=None,
                      stream=None, norm=None) -> None:
    """Chunked prefill over packed sequences.  q, k [T, H, dk], v [T, H, dv];
    g, beta [T, H] fp32; cu_seqlens [N+1] int32 (device); state_in
    [N, H, dv, dk] fp32 or None; state_out [N, H, dv, dk] fp32; o [T, H, dv];
    optional L_out / fixed_out [max_chunks, H, dv, dk], M_out [max_chunks, H,
    dk, dk] with max_chunks = gdr_max_chunks(T, N, chunk); M_out[c, h] is M_c
    with S_end = S_start @ M_c + L_c.  workspace: a uint8 device tensor of
    gdr_chunk_prefill_workspace_bytes(...) bytes, or None to allocate one here
    (on the launch stream, so that the caching allocator does not hand its
    memory to work on another stream while the kernels still use it).  norm: as
    gdr_decode_step's."""
    args, (T, N, H, dk, dv) = _prefill_args(q, k, v, g, beta, cu_seqlens, state_in, state_out, o,
                                            chunk, L_out, M_out, fixed_out, "gdr_chunk_prefill")
    dev = _device(q, "q")
    after = _norm_after(o, norm, dev, stream)
    if workspace is None:
        need = gdr_chunk_prefill_workspace_bytes(T, N, H, dk, dv, chunk, q.dtype)
        _, _, workspace = _workspace(None, max(need, 1), dev, stream)
    _launch("gdr_chunk_prefill", _load().gdr_chunk_prefill, dev, stream, *args,
            _dev_ptr(workspace, "workspace", (torch.uint8,)), workspace.numel())
    after()


def gdr_chunk_prefill_noalloc(q, k, v, g, beta, cu_seqlens, state_in, state_out, o, *, chunk=64,
                              L_out=None, M_out=None, fixed_out=None, stream=None,
                              norm=None) -> None:
    """gdr_chunk_prefill on the library's static device scratch: no workspace
    argument and no allocation, for callers that cannot allocate (e.g. under
    HIP graph capture).  Same arguments and results as gdr_chunk_prefill; a
    call that needs more than the scratch holds raises GdrError.  Calls that
    overlap on one device share the scratch and race."""
    args, _ = _prefill_args(q, k, v, g, beta, cu_seqlens, state_in, state_out, o, chunk, L_out,
                            M_out, fixed_out, "gdr_chunk_prefill_noalloc")
    dev = _device(q, "q")
    after = _norm_after(o, norm, dev, stream)
    _launch("gdr_chunk_prefill_noalloc", _load().gdr_chunk_prefill_noalloc, dev, stream, *args)
    after()


def gdr_state_fixup(L, M, state_in, chunk_offsets, fixed, stream=None) -> None:
    """fixed[c] = fixed[c-1] @ M_c + L_c over each sequence's chunk slots.
    L, fixed [n_chunks, H, dv, dk], M [n_chunks, H, dk, dk] fp32 (M[c, h] = M_c);
    state_in [N, H, dv, dk] fp32 or None; chunk_offsets [N+1] int32 (device)."""
    n_chunks, H, dv, dk = L.shape
    N = chunk_offsets.shape[0] - 1
    if M.shape != (n_chunks, H, dk, dk) or fixed.shape != L.shape or \
            (state_in is not None and state_in.shape != (N, H, dv, dk)):
        raise GdrError("gdr_state_fixup: inconsistent shapes")
    st = _load().gdr_state_fixup(
        _dev_ptr(L, "L", _F32), _dev_ptr(M, "M", _F32),
        _dev_ptr(state_in, "state_in", _F32, optional=True),
        _dev_ptr(chunk_offsets, "chunk_offsets", _I32), N, _dev_ptr(fixed, "fixed", _F32),
        n_chunks, H, dk, dv, _stream(stream))
    _check(st, "gdr_state_fixup")


# A single token's call costs about as much on the host as on the GPU: the current
# stream is read as a raw handle and the device is switched only when it has to be.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _device(t, name):
    """Index of the GPU that holds t."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0 or not t.is_cuda:
        raise GdrError(f"{name} must be a torch tensor on the GPU")
    return dev


def _ptr(t, name, dtypes, dev):
    """Pointer of a contiguous tensor on GPU `dev` (None: NULL)."""
    if t is None:
        return None
    if _device(t, name) != dev:
        raise GdrError(f"{name} is on another device than the first tensor")
    if not t.is_contiguous():
        raise GdrError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise GdrError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return t.data_ptr()


def _need(t, name):
    if t is None:
        raise GdrError(f"{name} is required")
    return t


def _rows_ptr(t, name, dev):
    """Pointer and token stride of a [tokens, heads, d] tensor whose tokens may
    be rows of a wider tensor (stride 0: dense)."""
    if t.is_contiguous():
        return _ptr(t, name, _IO, dev), 0
    if _device(t, name) != dev:
        raise GdrError(f"{name} is on another device than the first tensor")
    if t.dtype not in _IO:
        raise GdrError(f"{name} has dtype {t.dtype}, expected one of {_IO}")
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 or (h > 1 and sh != d) or (n > 1 and st < h * d):
        raise GdrError(f"{name}: the heads of a token must be contiguous and tokens must not overlap")
    return t.data_ptr(), st if n > 1 else 0


def _gates(g, tokens, H, dev, who):
    """Pointer and decay code of g, [tokens, H] or [H]."""
    if g.shape == (tokens, H):
        return _ptr(g, "g", _F32, dev), GDR_DECAY_TOKEN
    if g.shape == (H,):
        return _ptr(g, "g", _F32, dev), GDR_DECAY_HEAD
    raise GdrError(f"{who}: g must have shape {(tokens, H)} or {(H,)}")


def _workspace(workspace, need, dev, stream):
    """Pointer, size and tensor of the caller's workspace, or of one allocated
    here on the launch stream (none when none is needed)."""
    if workspace is None:
        if not need:
            return None, 0, None
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return _ptr(workspace, "workspace", (torch.uint8,), dev), workspace.numel(), workspace


def _launch(who, fn, dev, stream, *args):
    """fn(*args, stream) with GPU `dev` current; raises on a non-OK status."""
    handle = _raw_stream(dev) if stream is None else _stream(stream)
    if torch.cuda.current_device() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        _check(st, who)


def _same_dtype(who, names, first, *others):
    for t in others:
        if t.dtype != first.dtype:
            raise GdrError(f"{who}: {names} must share a dtype")


def gdr_linear_decode(q, k, v, g, state, o, *, scale=1.0, stream=None, norm=None) -> None:
    """One token of linear attention with a decay for each head, S <- e^g S +
    v k^T, o = scale S q, state updated in place.  q, k [N, Hk, dk], v [N, H,
    dv] (bf16 or fp32, one dtype; tokens may be rows of wider tensors); g [N, H]
    or [H] fp32; state [N, H, dv, dk] fp32; o [N, H, dv] bf16 or fp32.  Value
    head h reads query and key head h // (H // Hk).  norm: as gdr_decode_step's."""
    who = "gdr_linear_decode"
    N, Hk, dk = q.shape
    H, dv = v.shape[1:]
    if k.shape != q.shape or v.shape[0] != N or state.shape != (N, H, dv, dk) \
            or o.shape != (N, H, dv):
        raise GdrError(f"{who}: inconsistent shapes")
    _same_dtype(who, "q, k, v", q, k, v)
    dev = _device(q, "q")
    qp, qs = _rows_ptr(q, "q", dev)
    kp, ks = _rows_ptr(k, "k", dev)
    vp, vs = _rows_ptr(v, "v", dev)
    gp, decay = _gates(g, N, H, dev, who)
    after = _norm_after(o, norm, dev, stream)
    _launch(who, _load().gdr_linear_decode, dev, stream, qp, kp, vp, gp,
            _ptr(state, "state", _F32, dev), _ptr(o, "o", _IO, dev), N, H, Hk, dk, dv, qs, ks, vs,
            scale, decay, _code(q.dtype), _code(o.dtype))
    after()


def gdr_linear_prefill_workspace_bytes(T_total, N, H, dk, dv, in_dtype=GDR_BF16) -> int:
    """in_dtype: GDR_BF16 / GDR_FP32 or the torch dtype of q, k, v."""
    if isinstance(in_dtype, torch.dtype):
        in_dtype = _code(in_dtype)
    return int(_load().gdr_linear_prefill_workspace_bytes(T_total, N, H, dk, dv, in_dtype))


def gdr_linear_backward_workspace_bytes(T_total, N, H, Hk, dk, dv, in_dtype=GDR_BF16) -> int:
    """in_dtype: GDR_BF16 / GDR_FP32 or the torch dtype of q, k, v."""
    if isinstance(in_dtype, torch.dtype):
        in_dtype = _code(in_dtype)
    return int(_load().gdr_linear_backward_workspace_bytes(T_total, N, H, Hk, dk, dv, in_dtype))


def _linear_args(who, q, k, v, g, cu_seqlens, state_in, like_v):
    """Checks shared by prefill and backward; the device, the pointers of q, k,
    v, g, cu and state_in, the strides, the decay code and the sizes."""
    T, Hk, dk = q.shape
    H, dv = v.shape[1:]
    N = cu_seqlens.shape[0] - 1
    if k.shape != q.shape or v.shape[0] != T or cu_seqlens.dim() != 1 \
            or any(t.shape != (T, H, dv) for t in like_v):
        raise GdrError(f"{who}: inconsistent shapes")
    _same_dtype(who, "q, k, v", q, k, v)
    if state_in is not None and state_in.shape != (N, H, dv, dk):
        raise GdrError(f"{who}: state_in must have shape {(N, H, dv, dk)}")
    dev = _device(q, "q")
    qp, qs = _rows_ptr(q, "q", dev)
    kp, ks = _rows_ptr(k, "k", dev)
    vp, vs = _rows_ptr(v, "v", dev)
    gp, decay = _gates(g, T, H, dev, who)
    ptrs = (qp, kp, vp, gp, _ptr(_need(cu_seqlens, "cu_seqlens"), "cu_seqlens", _I32, dev), N,
            _ptr(state_in, "state_in", _F32, dev))
    return dev, ptrs, (qs, ks, vs), decay, (T, N, H, Hk, dk, dv)


def gdr_linear_prefill(q, k, v, g, cu_seqlens, state_in, state_out, o, *, scale=1.0,
                       workspace=None, stream=None, norm=None) -> None:
    """Linear attention with a decay for each head over packed sequences: S_t =
    e^g S_{t-1} + v_t k_t^T, o_t = scale S_t q_t.  q, k [T, Hk, dk], v [T, H, dv]
    (bf16 or fp32, one dtype; tokens may be rows of wider tensors); g [T, H] or
    [H] fp32; cu_seqlens [N+1] int32 (device); state_in [N, H, dv, dk] fp32 or
    None; state_out like it (may be state_in) or None; o [T, H, dv] bf16 or
    fp32.  workspace: as gdr_chunk_prefill's, by
    gdr_linear_prefill_workspace_bytes.  norm: as gdr_decode_step's (of rows
    behind the last sequence too, whose o is as the caller left it)."""
    who = "gdr_linear_prefill"
    dev, ptrs, strides, decay, (T, N, H, Hk, dk, dv) = _linear_args(who, q, k, v, g, cu_seqlens,
                                                                    state_in, (o,))
    if state_out is not None and state_out.shape != (N, H, dv, dk):
        raise GdrError(f"{who}: state_out must have shape {(N, H, dv, dk)}")
    after = _norm_after(o, norm, dev, stream)
    code, lib = _code(q.dtype), _load()
    wp, wb, workspace = _workspace(
        workspace, lib.gdr_linear_prefill_workspace_bytes(T, N, H, dk, dv, code), dev, stream)
    _launch(who, lib.gdr_linear_prefill, dev, stream, *ptrs,
            _ptr(state_out, "state_out", _F32, dev), _ptr(o, "o", _IO, dev), T, H, Hk, dk, dv,
            *strides, scale, decay, code, _code(o.dtype), wp, wb)
    after()


def gdr_linear_backward(q, k, v, g, cu_seqlens, state_in, do, dstate_out, dq, dk, dv, *, dg=None,
                        dstate_in=None, scale=1.0, workspace=None, stream=None) -> None:
    """Gradients of gdr_linear_prefill from do [T, H, dv] (the dtype of q) and
    dstate_out ([N, H, dv, dk] fp32 or None): dq, dk [T, Hk, dk] and dv [T, H,
    dv] (bf16 or fp32, one dtype), dg (fp32, the shape of g) and dstate_in
    ([N, H, dv, dk] fp32) where given.  workspace: by
    gdr_linear_backward_workspace_bytes."""
    who = "gdr_linear_backward"
    states = (cu_seqlens.shape[0] - 1, v.shape[1], v.shape[2], q.shape[2])
    if dq.shape != q.shape or dk.shape != q.shape or (dg is not None and dg.shape != g.shape) \
            or any(t is not None and t.shape != states for t in (dstate_out, dstate_in)):
        raise GdrError(f"{who}: inconsistent shapes")
    dev, ptrs, strides, decay, (T, N, H, Hk, kd, vd) = _linear_args(who, q, k, v, g, cu_seqlens,
                                                                    state_in, (do, dv))
    _same_dtype(who, "dq, dk, dv", dq, dk, dv)
    code, lib = _code(q.dtype), _load()
    wp, wb, workspace = _workspace(
        workspace, lib.gdr_linear_backward_workspace_bytes(T, N, H, Hk, kd, vd, code), dev, stream)
    _launch(who, lib.gdr_linear_backward, dev, stream, *ptrs, _ptr(do, "do", (q.dtype,), dev),
            _ptr(dstate_out, "dstate_out", _F32, dev), _ptr(dq, "dq", _IO, dev),
            _ptr(dk, "dk", _IO, dev), _ptr(dv, "dv", _IO, dev), _ptr(dg, "dg", _F32, dev),
            _ptr(dstate_in, "dstate_in", _F32, dev), T, H, Hk, kd, vd, *strides, scale, decay,
            code, _code(dq.dtype), wp, wb)


def _norm_args(who, x, w_after, gate, act, residual, w_before, like_x, outs):
    """Checks shared by the norm and its gradient: row operands like x, outputs
    of one dtype, weights [D] of one dtype.  Returns the device, rows, D and the
    codes of gate, input, weights and outputs."""
    shape = x.shape
    D = shape[-1] if shape else 0
    for t in (gate, residual, *like_x):
        if t is not None and (t.shape != shape or t.dtype != x.dtype):
            raise GdrError(f"{who}: row operands must have the shape and dtype of x")
    out = None
    for t in outs:
        if t is not None:
            out = t if out is None else out
            if t.shape != shape or t.dtype != out.dtype:
                raise GdrError(f"{who}: outputs must have the shape of x and one dtype")
    w = w_after if w_after is not None else w_before
    for t in (w_after, w_before):
        if t is not None and (t.shape != (D,) or t.dtype != w.dtype):
            raise GdrError(f"{who}: weights must have shape {(D,)} and one dtype")
    if gate is not None and act not in GDR_GATES:
        raise GdrError(f"{who}: act must be one of {sorted(GDR_GATES)}")
    return (_device(x, "x"), x.numel() // D if D else 0, D, GDR_GATES.get(act, 0), _code(x.dtype),
            GDR_FP32 if w is None else _code(w.dtype), GDR_FP32 if out is None else _code(out.dtype))


def gdr_block_norm(x, h=None, y=None, *, w_after=None, gate=None, act="silu", residual=None,
                   scale=1.0, w_before=None, eps=1e-6, stream=None) -> None:
    """Norms around a block with its gate and scaled residual, per row of x
    [..., D]: u = x / rms(x) * w_after, u *= act(gate), h = residual + scale * u,
    y = h / rms(h) * w_before, each part where its operand is given.  gate and
    residual like x; weights [D]; h and y [..., D] (h may be left out where y is
    wanted; y exactly with w_before).  bf16 or fp32 each."""
    dev, ptrs, rows, tail = _norm_call(x, h, y, w_after, gate, act, residual, scale, w_before, eps)
    _launch("gdr_block_norm", _load().gdr_block_norm, dev, stream, *ptrs, rows, *tail)


def _norm_call(x, h=None, y=None, w_after=None, gate=None, act="silu", residual=None, scale=1.0,
               w_before=None, eps=1e-6):
    """Device and arguments of a gdr_block_norm call: pointers, rows and the rest."""
    who = "gdr_block_norm"
    dev, rows, D, ac, ic, wc, oc = _norm_args(who, x, w_after, gate, act, residual, w_before, (),
                                              (h, y))
    return dev, (_ptr(x, "x", _IO, dev), _ptr(w_after, "w_after", _IO, dev),
                 _ptr(gate, "gate", _IO, dev), _ptr(residual, "residual", _IO, dev),
                 _ptr(w_before, "w_before", _IO, dev), _ptr(h, "h", _IO, dev),
                 _ptr(y, "y", _IO, dev)), rows, (D, scale, eps, ac, ic, wc, oc)


def _nothing():
    pass


def _norm_after(o, norm, dev, stream):
    """The call of gdr_block_norm on o that `norm` asks for, on the stream of the
    recurrence's launch on GPU `dev`, its arguments checked now: by the library too, in a call for no rows, which launches nothing, and the
    number of rows by the size of the gradient's workspace, 0 for rows that no norm
    takes."""
    if norm is None:
        return _nothing
    who, lib = "gdr_block_norm", _load()
    fn = lib.gdr_block_norm
    at, ptrs, rows, tail = _norm_call(o, **norm)
    if at != dev:
        raise GdrError("o is on another device than the first tensor")
    if norm.get("h") is None and norm.get("y") is None:
        raise GdrError(f"{who}: h or y is required")
    if (norm.get("y") is None) != (norm.get("w_before") is None):
        raise GdrError(f"{who}: y is given exactly when w_before is")
    _launch(who, fn, dev, stream, *ptrs, 0, *tail)
    if rows and not lib.gdr_block_norm_backward_workspace_bytes(rows, tail[0]):
        raise GdrError(f"{who}: rows={rows}")
    return lambda: _launch(who, fn, dev, stream, *ptrs, rows, *tail)


def gdr_block_norm_backward_workspace_bytes(rows, D) -> int:
    return int(_load().gdr_block_norm_backward_workspace_bytes(rows, D))


def gdr_block_norm_backward(x, dh, dy, dx, *, w_after=None, gate=None, act="silu", residual=None,
                            scale=1.0, w_before=None, eps=1e-6, dgate=None, dresidual=None,
                            dw_after=None, dw_before=None, workspace=None, stream=None) -> None:
    """Gradients of gdr_block_norm from dh and dy (like x; dh None: zero, dy
    exactly with w_before): dx, and dgate, dresidual (like x) and dw_after,
    dw_before ([D] fp32) where given.  workspace: a uint8 device tensor of
    gdr_block_norm_backward_workspace_bytes(rows, D) bytes, or None to allocate
    one here on the launch stream."""
    who = "gdr_block_norm_backward"
    if any(t is not None and t.shape != x.shape[-1:] for t in (dw_after, dw_before)):
        raise GdrError(f"{who}: weight gradients must have shape {tuple(x.shape[-1:])}")
    dev, rows, D, ac, ic, wc, oc = _norm_args(who, x, w_after, gate, act, residual, w_before,
                                              (dh, dy), (dx, dgate, dresidual))
    lib, need = _load(), 0
    if dw_after is not None or dw_before is not None:
        need = lib.gdr_block_norm_backward_workspace_bytes(rows, D)
    wp, wb, workspace = _workspace(workspace, need, dev, stream)
    _launch(who, lib.gdr_block_norm_backward, dev, stream, _ptr(x, "x", _IO, dev),
            _ptr(w_after, "w_after", _IO, dev), _ptr(gate, "gate", _IO, dev),
            _ptr(residual, "residual", _IO, dev), _ptr(w_before, "w_before", _IO, dev),
            _ptr(dh, "dh", _IO, dev), _ptr(dy, "dy", _IO, dev), _ptr(dx, "dx", _IO, dev),
            _ptr(dgate, "dgate", _IO, dev), _ptr(dresidual, "dresidual", _IO, dev),
            _ptr(dw_after, "dw_after", _F32, dev), _ptr(dw_before, "dw_before", _F32, dev),
            rows, D, scale, eps, ac, ic, wc, oc, wp, wb)
