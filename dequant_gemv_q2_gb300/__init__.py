"""Fused dequantize-plus-matvec over packed ~2-bit weights on GB300.

Thin ctypes binding of ``libq2.so`` (``include/q2.h``): the functions below
carry the C names and only marshal arguments; every step of y = W x runs in
the library's CUDA kernels.  PyTorch is used for device memory and streams.
Importing works without a GPU; calling a compute entry point without the
built library raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from . import build as _build

FP16, BPDQ, TRELLIS, LEECH, NOWEIGHTS, INT4 = 0, 1, 2, 3, 4, 5
FMT_NAMES = {FP16: "fp16", BPDQ: "bpdq", TRELLIS: "trellis", LEECH: "leech", NOWEIGHTS: "noweights", INT4: "int4"}
EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -7
ERR_LENGTH, ERR_PAGE = 0x100, 0x200     # bits of device_errors()
MAX_NTOK = 64
INV_SQRT8_F32 = float(np.float32(1.0 / np.sqrt(8.0)))

_lib = None


class Q2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {q2_strerror(status)} ({status})")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libq2.so (build it first if asked); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        if not build_if_missing:
            raise RuntimeError(f"libq2.so not built ({_build.LIB}); run __graft_entry__.build()")
        _build.build()
    L = ctypes.CDLL(_build.LIB)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    psz = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "q2_pack_fp16": [vp, i32, i32, vp, psz],
        "q2_pack_bpdq": [vp, vp, vp, i32, i32, vp, psz],
        "q2_pack_trellis": [vp, vp, vp, i32, i32, vp, psz],
        "q2_pack_leech": [vp, vp, vp, i32, i32, ctypes.c_float, i32, vp, psz],
        "q2_pack_int4": [vp, vp, vp, i32, i32, i32, vp, psz],
        "q2_pack_noweights": [i32, i32, vp, psz],
        "q2_bind": [vp, vp, ctypes.POINTER(vp)],
        "q2_workspace_bytes": [vp, i32, psz],
        "q2_set_workspace": [vp, vp, sz],
        "q2_info": [vp, ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)],
        "q2_bytes": [vp, i32, psz],
        "q2_gemv": [i32, vp, vp, vp, i32, vp],
        "q2_gemv_x8": [vp, vp, vp, vp, i32, vp],
        "q2_rmsnorm": [vp, ctypes.c_longlong, i32, i32, i32, vp, vp, vp, ctypes.c_float, vp, ctypes.c_longlong, vp, vp, vp],
        "q2_attend_workspace_bytes": [i32, i32, i32, i32, psz],
        "q2_attend": [vp, vp, ctypes.c_longlong, vp, vp, ctypes.c_longlong, vp, i32, i32, ctypes.c_float, vp,
                      ctypes.c_longlong, vp, sz, vp],
        "q2_decode_bytes": [vp, psz],
        "q2_decode": [vp, vp, vp],
        "q2_gemv_chain": [i32, vp, vp, vp, vp, i32, i32, vp],
        "q2_gemv_bpdq_noalloc": [vp, vp, vp, vp],
        "q2_device_errors": [ctypes.POINTER(ctypes.c_uint)],
        "q2_debug_wait_limit": [ctypes.c_longlong],
        "q2_rotate": [vp, vp, i32, i32, i32, vp, vp, vp],
        "q2_rotate_split": [i32, ctypes.POINTER(i32), ctypes.POINTER(i32)],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = i32
    L.q2_unbind.argtypes = [vp]
    L.q2_unbind.restype = None
    L.q2_strerror.argtypes = [i32]
    L.q2_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


EXPORTS = ["q2_pack_fp16", "q2_pack_bpdq", "q2_pack_trellis", "q2_pack_leech", "q2_pack_int4", "q2_pack_noweights",
           "q2_bind", "q2_unbind", "q2_workspace_bytes", "q2_set_workspace", "q2_info", "q2_bytes",
           "q2_gemv", "q2_gemv_chain", "q2_gemv_x8", "q2_rmsnorm",
           "q2_attend", "q2_attend_workspace_bytes", "q2_decode_bytes", "q2_decode", "q2_strerror", "q2_gemv_bpdq_noalloc",
           "q2_device_errors", "q2_debug_wait_limit", "q2_rotate", "q2_rotate_split"]


def q2_strerror(status: int) -> str:
    try:
        return load().q2_strerror(int(status)).decode()
    except Exception:  # library missing: still give a message
        return f"status {status}"


def _ptr(a: np.ndarray):
    return ctypes.c_void_p(a.ctypes.data) if a is not None else None


def _check(st: int, where: str) -> None:
    if st != 0:
        raise Q2Error(st, where)


def _pack(fn, args, where: str) -> np.ndarray:
    L = load()
    n = ctypes.c_size_t(0)
    _check(getattr(L, fn)(*args, None, ctypes.byref(n)), where)
    out = np.zeros(n.value, dtype=np.uint8)
    _check(getattr(L, fn)(*args, _ptr(out), ctypes.byref(n)), where)
    return out


def q2_pack_fp16(w: np.ndarray) -> np.ndarray:
    w = np.ascontiguousarray(w, dtype=np.float16)
    R, C = w.shape
    return _pack("q2_pack_fp16", [_ptr(w.view(np.uint16)), R, C], "q2_pack_fp16")


def q2_pack_bpdq(plane0: np.ndarray, plane1: np.ndarray, coef: np.ndarray) -> np.ndarray:
    p0 = np.ascontiguousarray(plane0, dtype=np.uint8)
    p1 = np.ascontiguousarray(plane1, dtype=np.uint8)
    cf = np.ascontiguousarray(coef, dtype=np.float16)
    R, C = p0.shape[0], p0.shape[1] * 8
    return _pack("q2_pack_bpdq", [_ptr(p0), _ptr(p1), _ptr(cf.view(np.uint16)), R, C], "q2_pack_bpdq")


def q2_pack_trellis(stream: np.ndarray, table: np.ndarray, scale: np.ndarray) -> np.ndarray:
    st = np.ascontiguousarray(stream, dtype=np.uint8)
    tb = np.ascontiguousarray(table, dtype=np.float16)
    sc = np.ascontiguousarray(scale, dtype=np.float16)
    R, C = st.shape[0], st.shape[1] * 256
    return _pack("q2_pack_trellis", [_ptr(st), _ptr(tb.view(np.uint16)), _ptr(sc.view(np.uint16)), R, C],
                 "q2_pack_trellis")


LEECH_PLANES3, LEECH_OFFSET4 = 0, 1


def q2_pack_leech(v: np.ndarray, tail: np.ndarray, scale: np.ndarray, C: int, layout: int = LEECH_PLANES3) -> np.ndarray:
    vv = np.ascontiguousarray(v, dtype=np.int8)
    tl = np.ascontiguousarray(tail, dtype=np.float16)
    sc = np.ascontiguousarray(scale, dtype=np.float16)
    R = vv.shape[0]
    tptr = _ptr(tl.view(np.uint16)) if tl.size else None
    return _pack("q2_pack_leech", [_ptr(vv), tptr, _ptr(sc.view(np.uint16)), R, C,
                                   ctypes.c_float(INV_SQRT8_F32), int(layout)], "q2_pack_leech")


def q2_pack_int4(code: np.ndarray, scale: np.ndarray, zero=None, group: int = 128) -> np.ndarray:
    """code: uint8 [R][C/2] (low four bits: even column); scale: fp16 [R][C/group]; zero: uint8 of that shape or None (8)."""
    cd = np.ascontiguousarray(code, dtype=np.uint8)
    sc = np.ascontiguousarray(scale, dtype=np.float16)
    zr = None if zero is None else np.ascontiguousarray(zero, dtype=np.uint8)
    R, C = cd.shape[0], cd.shape[1] * 2
    if group in (32, 64, 128) and C % group == 0:
        for a, what in ((sc, "scale"), (zr, "zero")):
            if a is not None and a.shape != (R, C // group):
                raise Q2Error(ESHAPE, f"q2_pack_int4: {what} is {a.shape}, not {(R, C // group)}")
    return _pack("q2_pack_int4", [_ptr(cd), _ptr(sc.view(np.uint16)), _ptr(zr), R, C, int(group)], "q2_pack_int4")


def q2_pack_noweights(R: int, C: int) -> np.ndarray:
    return _pack("q2_pack_noweights", [R, C], "q2_pack_noweights")


def _stream_ptr(stream):
    """The cudaStream_t of a torch stream, or of the current one (asked for without making a stream object: 0.15
    instead of 3.2 us per call on the GB300's host cores; by the public call where torch has no such functions)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    except AttributeError:
        return torch.cuda.current_stream().cuda_stream


def _check_tensor(where: str, name: str, t, dtype, shape, strides=None) -> None:
    """Refuse a tensor that the C call would misread: another type, shape or (row-major unless `strides`) layout, or not on a GPU."""
    if t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous():
        return
    if t.dtype is not dtype or not t.is_cuda:
        raise Q2Error(EINVAL, f"{where}: {name} is {t.dtype} on {t.device}, not {dtype} on a GPU")
    if t.shape != shape:
        raise Q2Error(ESHAPE, f"{where}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous() and (strides is None or any(n > 1 and a != b for n, a, b in zip(shape, t.stride(), strides))):
        raise Q2Error(ESHAPE, f"{where}: {name} has strides {t.stride()}")


def _check_rows(where: str, name: str, t, ntok: int, width: int) -> None:
    """Refuse what the C call would not read (or write) as fp16 [ntok][width]: rows of another width, fewer of them,
    another type or layout, or a tensor that is not on a GPU.  Rows behind the first ntok are left alone."""
    import torch
    if t.dtype is not torch.float16 or not t.is_cuda:
        raise Q2Error(EINVAL, f"{where}: {name} is {t.dtype} on {t.device}, not {torch.float16} on a GPU")
    if t.numel() != ntok * width and not (t.dim() == 2 and t.shape[0] >= ntok and t.shape[1] == width):
        raise Q2Error(ESHAPE, f"{where}: {name} has shape {tuple(t.shape)}, not {(ntok, width)}")
    if not t.is_contiguous():
        raise Q2Error(ESHAPE, f"{where}: {name} has strides {t.stride()}")


def _new(make, shape, dtype, device, stream):
    """A tensor made on the stream that writes it: memory of another stream's might still be in that one's use."""
    import torch
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _zero_workspace(n: int, device):
    """A workspace of zeros, filled when this returns: its first call may come on any stream."""
    import torch
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    if ws.is_cuda and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(ws.device).synchronize()
    return ws


def _workspace_bytes(where: str, ws) -> int:
    """The bytes of a workspace, which is one run of GPU memory."""
    if not ws.is_cuda:
        raise Q2Error(EINVAL, f"{where}: workspace on {ws.device}, not on a GPU")
    if not ws.is_contiguous():
        raise Q2Error(ESHAPE, f"{where}: workspace has strides {ws.stride()}")
    return ws.numel() * ws.element_size()


def device_errors() -> int:
    """The tensor-core and attention kernels' device error word (then cleared); 0 is normal."""
    v = ctypes.c_uint(0)
    _check(load().q2_device_errors(ctypes.byref(v)), "q2_device_errors")
    return v.value


def debug_wait_limit(polls: int) -> None:
    """Test hook: limit the tensor-core kernel's stage waits to `polls` polls (0 = normal)."""
    _check(load().q2_debug_wait_limit(int(polls)), "q2_debug_wait_limit")


class Packed:
    """A packed matrix bound to its device copy (and a split-K workspace).

    ``blob`` is the host blob from a ``q2_pack_*`` call.  The device copy and
    the workspace are torch tensors owned by this object.
    """

    def __init__(self, blob: np.ndarray, device="cuda", ntok_max: int = MAX_NTOK, workspace=None):
        import torch
        L = load()
        self.blob = blob
        self.dev = torch.from_numpy(blob).to(device)
        assert self.dev.data_ptr() % 256 == 0
        h = ctypes.c_void_p()
        _check(L.q2_bind(_ptr(blob), ctypes.c_void_p(self.dev.data_ptr()), ctypes.byref(h)), "q2_bind")
        self.h = h
        f, R, C = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _check(L.q2_info(h, ctypes.byref(f), ctypes.byref(R), ctypes.byref(C)), "q2_info")
        self.fmt, self.R, self.C = f.value, R.value, C.value
        self._fn, self._f16 = L.q2_gemv, torch.float16
        self.ws = None
        # the workspace of every call up to ntok_max tokens (the paths differ by token count)
        need = max(self.workspace_bytes(t) for t in range(1, int(ntok_max) + 1))
        if workspace is not None:
            self.set_workspace(workspace)
        elif need:
            self.set_workspace(_zero_workspace(need, device))

    def workspace_bytes(self, ntok: int) -> int:
        n = ctypes.c_size_t(0)
        _check(load().q2_workspace_bytes(self.h, int(ntok), ctypes.byref(n)), "q2_workspace_bytes")
        return n.value

    def set_workspace(self, ws) -> None:
        n = _workspace_bytes("q2_set_workspace", ws)
        _check(load().q2_set_workspace(self.h, ctypes.c_void_p(ws.data_ptr()), n), "q2_set_workspace")
        self.ws = ws

    def bytes_read(self, ntok: int = 1) -> int:
        n = ctypes.c_size_t(0)
        _check(load().q2_bytes(self.h, int(ntok), ctypes.byref(n)), "q2_bytes")
        return n.value

    def gemv(self, x, y=None, stream=None, fmt=None):
        """y[ntok][R] = x[ntok][C] @ W^T through q2_gemv (asynchronous).

        x and y: fp16, contiguous, on the GPU; a token's C columns may be of any shape ([ntok][heads][dim]).
        """
        f16, C, R, shape = self._f16, self.C, self.R, x.shape
        if len(shape) == 1:
            x = x.view(1, -1)
            shape = x.shape
        ntok = shape[0]
        # what each tensor has to be is tested here at once, and put into words by the function called otherwise
        if not (x.dtype is f16 and x.is_cuda and shape == (ntok, C) and x.is_contiguous()):
            _check_rows("q2_gemv", "x", x, ntok, C)
        if y is None:
            import torch
            y = _new(torch.empty, (ntok, R), f16, x.device, stream)
        elif not (y.dtype is f16 and y.is_cuda and y.shape == (ntok, R) and y.is_contiguous()):
            _check_rows("q2_gemv", "y", y, ntok, R)
        st = self._fn(self.fmt if fmt is None else int(fmt), self.h, x.data_ptr(), y.data_ptr(), ntok, _stream_ptr(stream))
        if st:
            raise Q2Error(st, "q2_gemv")
        return y

    def gemv_x8(self, x8, xscale, y=None, stream=None):
        """y[ntok][R] = xscale[ntok] * (x8[ntok][C] @ W^T) through q2_gemv_x8 (INT4 weights; asynchronous)."""
        import torch
        if x8.dim() == 1:
            x8 = x8.view(1, -1)
        shape = x8.shape
        ntok = shape[0]
        # what each tensor has to be is tested here at once, and put into words by the function called otherwise
        if not (x8.dtype is torch.int8 and x8.is_cuda and shape[1:] == (self.C,) and x8.is_contiguous()):
            _check_tensor("q2_gemv_x8", "x8", x8, torch.int8, (ntok, self.C))
        if not (xscale.dtype is torch.float32 and xscale.is_cuda and xscale.shape == (ntok,) and xscale.is_contiguous()):
            _check_tensor("q2_gemv_x8", "xscale", xscale, torch.float32, (ntok,))
        if y is None:
            y = _new(torch.empty, (ntok, self.R), torch.float16, x8.device, stream)
        elif not (y.dtype is torch.float16 and y.is_cuda and y.shape == (ntok, self.R) and y.is_contiguous()):
            _check_tensor("q2_gemv_x8", "y", y, torch.float16, (ntok, self.R))
        st = load().q2_gemv_x8(self.h, x8.data_ptr(), xscale.data_ptr(), y.data_ptr(), ntok, _stream_ptr(stream))
        if st:
            raise Q2Error(st, "q2_gemv_x8")
        return y

    def decode(self, stream=None):
        """Canonical decode on the device (a uint8 tensor of q2_decode_bytes)."""
        import torch
        n = ctypes.c_size_t(0)
        _check(load().q2_decode_bytes(self.h, ctypes.byref(n)), "q2_decode_bytes")
        out = _new(torch.zeros, n.value, torch.uint8, self.dev.device, stream)
        _check(load().q2_decode(self.h, ctypes.c_void_p(out.data_ptr()), _stream_ptr(stream)), "q2_decode")
        return out

    def close(self) -> None:
        if getattr(self, "h", None):
            load().q2_unbind(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def q2_gemv(fmt: int, packed: Packed, x, y, ntok: int, stream=None) -> int:
    """The C entry point with its own argument order (status returned)."""
    return load().q2_gemv(int(fmt), packed.h, ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(y.data_ptr()),
                          int(ntok), _stream_ptr(stream))


class Chain:
    """A decode step's chain of GEMVs run through q2_gemv_chain.

    ``links`` is a list of (Packed, x, y) with device fp16 tensors x [ntok][C]
    and y [ntok][R]; the pointer arrays are built once, so ``run`` only makes
    the one C call (and may be captured in a CUDA graph).
    """

    def __init__(self, links, ntok: int, lookahead: int = 2):
        n = len(links)
        self.links = list(links)            # keeps the tensors alive
        self.ntok, self.lookahead = int(ntok), int(lookahead)
        for i, (p, x, y) in enumerate(self.links):
            _check_rows("q2_gemv_chain", f"x of link {i}", x, self.ntok, p.C)
            _check_rows("q2_gemv_chain", f"y of link {i}", y, self.ntok, p.R)
        self._fmt = (ctypes.c_int * n)(*[p.fmt for p, _, _ in links])
        self._h = (ctypes.c_void_p * n)(*[p.h.value for p, _, _ in links])
        self._x = (ctypes.c_void_p * n)(*[x.data_ptr() for _, x, _ in links])
        self._y = (ctypes.c_void_p * n)(*[y.data_ptr() for _, _, y in links])

    def run(self, stream=None) -> None:
        st = load().q2_gemv_chain(len(self.links), self._fmt, self._h, self._x, self._y, self.ntok, self.lookahead,
                                  _stream_ptr(stream))
        _check(st, "q2_gemv_chain")


def q2_rotate_split(C: int) -> tuple:
    """(nh, nq) of the page's examples: nh = 2048 if it divides C, else 1024."""
    nh, nq = ctypes.c_int(), ctypes.c_int()
    _check(load().q2_rotate_split(int(C), ctypes.byref(nh), ctypes.byref(nq)), "q2_rotate_split")
    return nh.value, nq.value


def q2_rotate(x, x_rot, ntok: int, C: int, nh: int, signs, q, stream=None) -> int:
    """The C entry point (status returned): x_rot = (H (x) Q)(S x) per token."""
    return load().q2_rotate(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(x_rot.data_ptr()), int(ntok), int(C),
                            int(nh), ctypes.c_void_p(signs.data_ptr()),
                            ctypes.c_void_p(q.data_ptr()) if q is not None else None, _stream_ptr(stream))


class Rotation:
    """The activation rotation of one input width, x_rot = (H (x) Q)(S x).

    ``signs``: uint8 [ceil(C/8)] column sign bits; ``q``: fp32 [nq][nq]
    (None when nq == 1).  Both are copied to the device once.
    """

    def __init__(self, signs: np.ndarray, q, nh: int, C: int, device="cuda"):
        import torch
        self.C, self.nh = int(C), int(nh)
        self.signs = torch.from_numpy(np.ascontiguousarray(signs, dtype=np.uint8)).to(device)
        self.q = None if q is None else torch.from_numpy(np.ascontiguousarray(q, dtype=np.float32)).to(device)

    def apply(self, x, out=None, stream=None):
        """Rotate x [ntok][C] (fp16, device) into a new or given fp16 tensor (asynchronous)."""
        import torch
        if x.dim() == 1:
            x = x.view(1, -1)
        _check_rows("q2_rotate", "x", x, x.shape[0], self.C)
        if out is None:
            out = _new(torch.empty, x.shape, x.dtype, x.device, stream)
        else:
            _check_rows("q2_rotate", "out", out, x.shape[0], self.C)
        _check(q2_rotate(x, out, x.shape[0], self.C, self.nh, self.signs, self.q, stream), "q2_rotate")
        return out


class RmsNorm:
    """Root-mean-square norm of rows with the residual's addition in front and
    an fp16 and/or an 8-bit output behind it (``q2_rmsnorm``).

    ``weight``: fp16 [C] (numpy, or a torch tensor kept on its device).
    """

    def __init__(self, weight, eps: float = 1e-6, device="cuda"):
        import torch
        w = weight if isinstance(weight, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(weight)).to(device)
        _check_tensor("RmsNorm", "weight", w, torch.float16, (w.numel(),))
        self.weight, self.eps, self.C, self._w = w, float(eps), w.numel(), w.data_ptr()
        self._fn, self._f16 = load().q2_rmsnorm, torch.float16

    def _ld(self, name: str, t, shape, heads: int) -> int:
        """The token stride of fp16 rows [ntok][heads][C] of which each token's are contiguous."""
        import torch
        if not (t.dtype is torch.float16 and t.is_cuda and t.shape == shape):
            _check_tensor("q2_rmsnorm", name, t, torch.float16, shape)
        if t.is_contiguous():
            return heads * self.C
        st = t.stride()
        if (self.C > 1 and st[-1] != 1) or (heads > 1 and st[1] != self.C):
            raise Q2Error(ESHAPE, f"q2_rmsnorm: {name} has strides {st}")
        return st[0] if shape[0] > 1 else heads * self.C

    def apply(self, x, residual=None, residual_out=None, out=None, out8=None, scale8=None, stream=None):
        """Norm of the rows x [ntok][C] or [ntok][heads][C] (fp16; a token's rows contiguous, any token stride).

        ``residual`` (fp16, of x's shape, contiguous) is added first; the sum goes to ``residual_out`` (default:
        back to ``residual``).  ``out``: fp16 of x's shape, laid out as x may be (x itself included); made here when
        neither ``out`` nor ``out8`` is given.  ``out8`` (int8, x's shape) and ``scale8`` (fp32, a scale per row)
        take the 8-bit output.  Returns ``out`` (asynchronous).
        """
        f16, C, shape = self._f16, self.C, x.shape
        dims = len(shape)
        if dims not in (2, 3) or shape[-1] != C:
            raise Q2Error(ESHAPE, f"q2_rmsnorm: x has shape {tuple(shape)}, not [ntok][{C}] or [ntok][heads][{C}]")
        ntok, heads = shape[0], shape[1] if dims == 3 else 1
        ldx = ldy = heads * C
        # what each tensor has to be is tested here at once, and put into words by the functions called otherwise
        if not (x.dtype is f16 and x.is_cuda and x.is_contiguous()):
            ldx = self._ld("x", x, shape, heads)
        y = y8 = s8 = r = ro = None
        if out is not None:
            if not (out.dtype is f16 and out.is_cuda and out.shape == shape and out.is_contiguous()):
                ldy = self._ld("out", out, shape, heads)
            y = out.data_ptr()
        elif out8 is None:
            import torch
            out = _new(torch.empty, shape, f16, x.device, stream)
            y = out.data_ptr()
        if residual is not None:
            if not (residual.dtype is f16 and residual.is_cuda and residual.shape == shape and residual.is_contiguous()):
                _check_tensor("q2_rmsnorm", "residual", residual, f16, shape)
            ro = r = residual.data_ptr()
        if residual_out is not None:
            if not (residual_out.dtype is f16 and residual_out.is_cuda and residual_out.shape == shape
                    and residual_out.is_contiguous()):
                _check_tensor("q2_rmsnorm", "residual_out", residual_out, f16, shape)
            ro = residual_out.data_ptr()
        if out8 is not None:
            import torch
            _check_tensor("q2_rmsnorm", "out8", out8, torch.int8, shape)
            if scale8 is None:
                raise Q2Error(EINVAL, "q2_rmsnorm: out8 needs scale8")
            _check_tensor("q2_rmsnorm", "scale8", scale8, torch.float32, shape[:-1])
            y8, s8 = out8.data_ptr(), scale8.data_ptr()
        st = self._fn(x.data_ptr(), ldx, ntok, heads, C, r, ro, self._w, self.eps, y, ldy, y8, s8, _stream_ptr(stream))
        if st:
            raise Q2Error(st, "q2_rmsnorm")
        return out


class _KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong), ("npages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong), ("max_pages", ctypes.c_int)]


def _rows(name: str, t, shape) -> int:
    """The leading dimension of fp16 rows [batch][heads][dim], each sequence's contiguous."""
    import torch
    stride = t.stride()
    if not (t.dtype is torch.float16 and t.is_cuda and t.shape == shape and stride[1] == shape[2] and stride[2] == 1):
        _check_tensor("q2_attend", name, t, torch.float16, shape, (t.stride(0), shape[2], 1))
    return stride[0] if shape[0] > 1 else shape[1] * shape[2]


class PagedKV:
    """A paged key-value cache and attention of one new token per sequence over it (``q2_attend``).

    ``k``, ``v``: fp16 pools seen as [pages][page_size][kv_heads][dim], in any order of storage (dim contiguous; both
    alike).  ``table``: int32 [batch][max_pages] page numbers on the same GPU.  The tensors stay the caller's: pages,
    table and lengths may be changed between calls.  ``workspace``: uint8, zero when first used (made here if None).
    """

    def __init__(self, k, v, table, q_heads: int, workspace=None):
        import torch
        if k.dim() != 4 or table.dim() != 2:
            raise Q2Error(ESHAPE, "PagedKV: k is not [pages][page_size][kv_heads][dim], or table not [batch][max_pages]")
        if k.stride(3) != 1 and k.shape[3] > 1:
            raise Q2Error(ESHAPE, f"PagedKV: k has strides {k.stride()}")
        for name, t in (("k", k), ("v", v)):
            _check_tensor("PagedKV", name, t, torch.float16, k.shape, k.stride())
        if v.stride() != k.stride():
            raise Q2Error(ESHAPE, f"PagedKV: k has strides {k.stride()}, v {v.stride()}")
        _check_tensor("PagedKV", "table", table, torch.int32, table.shape, (table.stride(0), 1))
        self.k, self.v, self.table, self.q_heads = k, v, table, int(q_heads)
        pages, page, self.kv_heads, self.dim = k.shape
        self.batch = table.shape[0]
        self.scale = self.dim ** -0.5
        self._qshape = torch.Size((self.batch, self.q_heads, self.dim))
        self._kvshape = torch.Size((self.batch, self.kv_heads, self.dim))
        self._fn, self._f16, self._i32 = load().q2_attend, torch.float16, torch.int32
        self._kv = _KV(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), pages, page, self.kv_heads,
                       self.dim, table.data_ptr(), table.stride(0) if self.batch > 1 else table.shape[1], table.shape[1])
        self._ref = ctypes.byref(self._kv)
        n = ctypes.c_size_t(0)
        _check(load().q2_attend_workspace_bytes(self.batch, self.q_heads, self.kv_heads, self.dim, ctypes.byref(n)),
               "q2_attend_workspace_bytes")
        if workspace is None:
            workspace = _zero_workspace(n.value, k.device)
        size = _workspace_bytes("PagedKV", workspace)
        if size < n.value:
            raise Q2Error(EWORKSPACE, f"PagedKV: workspace of {size} bytes, {n.value} needed")
        self.ws, self._ws, self._ws_bytes = workspace, workspace.data_ptr(), size

    def attend(self, q, lens, new_k=None, new_v=None, scale=None, out=None, stream=None):
        """Attention of q [batch][q_heads][dim] over the first lens[b] (int32) tokens of each sequence.

        ``new_k``, ``new_v`` [batch][kv_heads][dim]: the new token's, counted by ``lens``; they are stored as token
        lens[b] - 1.  q, new_k, new_v and ``out`` may have any batch stride (slices of a projection's output).
        ``scale``: dim ** -0.5 if None.  Returns ``out`` (asynchronous).
        """
        f16, shape = self._f16, self._qshape
        # what each tensor has to be is tested here at once, and put into words by the functions called otherwise
        if out is None:
            import torch
            out = _new(torch.empty, shape, f16, q.device, stream)
        ldq = ldo = self.q_heads * self.dim
        if not (q.dtype is f16 and q.is_cuda and q.shape == shape and q.is_contiguous()):
            ldq = _rows("q", q, shape)
        if not (out.dtype is f16 and out.is_cuda and out.shape == shape and out.is_contiguous()):
            ldo = _rows("out", out, shape)
        if not (lens.dtype is self._i32 and lens.is_cuda and lens.shape == shape[:1] and lens.is_contiguous()):
            _check_tensor("q2_attend", "lens", lens, self._i32, shape[:1])
        nk = nv = None
        ldn = 0
        if new_k is not None and new_v is not None:
            shape = self._kvshape
            ldn = _rows("new_k", new_k, shape)
            if not (new_v.dtype is f16 and new_v.is_cuda and new_v.shape == shape and new_v.stride() == new_k.stride()):
                if _rows("new_v", new_v, shape) != ldn:
                    raise Q2Error(ESHAPE, "q2_attend: new_k and new_v have different batch strides")
            nk, nv = new_k.data_ptr(), new_v.data_ptr()
        elif new_k is not None or new_v is not None:
            raise Q2Error(EINVAL, "q2_attend: new_k and new_v go together")
        st = self._fn(self._ref, q.data_ptr(), ldq, nk, nv, ldn, lens.data_ptr(), self.batch, self.q_heads,
                      self.scale if scale is None else scale, out.data_ptr(), ldo, self._ws, self._ws_bytes,
                      _stream_ptr(stream))
        if st:
            raise Q2Error(st, "q2_attend")
        return out
