"""ctypes binding of the layers on irreps rows (include/cgtp_layers.h): group
norm with its activation, cross attention to a context, dropout.

As clebsch_gordan_tensor_amd.cgtp: this module checks shapes, dtypes and
devices, allocates outputs and workspaces with torch when the caller passes
none, and forwards raw pointers and the current stream. Every computation runs
in the HIP kernels of libcgtp.so.
"""

import ctypes

import numpy as np

from .cgtp import (_DT, _check, _lib, _need, _ptr, _stream, _torch, _torch_dtype, _vp, _ws_bytes, F64)

_i64, _size = ctypes.c_int64, ctypes.c_size_t
_i64p, _sizep, _vpp = ctypes.POINTER(_i64), ctypes.POINTER(_size), ctypes.POINTER(_vp)
_dbl, _u64, _u32 = ctypes.c_double, ctypes.c_uint64, ctypes.c_uint32

_SIGS = {
    "cgtp_samples_create": [_i64, _i64p, _vpp],
    "cgtp_samples_destroy": [_vp],
    "cgtp_norm_create": [ctypes.c_char_p, _i64, ctypes.c_int, _dbl, ctypes.c_int, _vpp],
    "cgtp_norm_destroy": [_vp],
    "cgtp_norm_query": [_vp, _i64p, _i64p, _i64p, _i64p],
    "cgtp_norm_workspace_size": [_vp, _vp, _sizep],
    "cgtp_norm_forward": [_vp] * 8 + [_size, _vp],
    "cgtp_norm_backward": [_vp] * 11 + [_size, _vp],
    "cgtp_dropout_create": [ctypes.c_char_p, ctypes.c_int, _vpp],
    "cgtp_dropout_destroy": [_vp],
    "cgtp_dropout_query": [_vp, _i64p],
    "cgtp_dropout_forward": [_vp, _i64, _vp, _dbl, _u64, _u32, _vp, _vp, _vp],
    "cgtp_dropout_backward": [_vp, _i64, _vp, _dbl, _u64, _u32, _vp, _vp],
}
for _name, _args in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int

EXPORTED = tuple(_SIGS)

_ACT = {"none": 0, "silu": 1, "gelu": 2}


def _acc_dtype(code):
    t = _torch()
    return t.float64 if code == F64 else t.float32


def _workspace(ws, nbytes, device):
    """(tensor, bytes) of the caller's workspace or a new one."""
    if ws is None:
        ws = _torch().empty(max(nbytes, 1), dtype=_torch().uint8, device=device)
    return ws, _ws_bytes(ws)


class _Handle:
    """An opaque handle of the library, destroyed with this object."""

    _h = None

    def _own(self, handle, destroy):
        self._h, self._destroy = handle, getattr(_lib, destroy)

    def __del__(self):
        if self._h and _lib is not None:
            self._destroy(self._h)
            self._h = None


class Samples(_Handle):
    """Rows of samples laid end to end: sample s owns rows ptr[s]..ptr[s+1]-1
    (cgtp_samples_create). ``ptr`` is a sequence, array or tensor of S + 1
    offsets; it is read on the host."""

    def __init__(self, ptr):
        if hasattr(ptr, "detach"):
            ptr = ptr.detach().cpu().numpy()
        ptr = np.asarray(ptr)
        if ptr.ndim != 1 or ptr.size < 1 or (ptr.size and not np.issubdtype(ptr.dtype, np.integer)):
            raise ValueError("ptr must be a one-dimensional array of S + 1 whole numbers")
        self.ptr = np.ascontiguousarray(ptr, np.int64)
        self.S, self.rows = len(self.ptr) - 1, int(self.ptr[-1])
        h = _vp()
        _check(_lib.cgtp_samples_create(self.S, self.ptr.ctypes.data_as(_i64p), ctypes.byref(h)),
               "cgtp_samples_create")
        self._own(h, "cgtp_samples_destroy")


class GroupNorm(_Handle):
    """Group norm of irreps rows with the activation of the even scalars
    (cgtp_norm_create); ``activation`` is "none", "silu" or "gelu"."""

    def __init__(self, irreps, groups, activation="none", eps=1e-5, dtype="f32"):
        self.irreps, self.groups, self.activation, self.eps = irreps, int(groups), activation, float(eps)
        self.dtype_code = _DT[dtype]
        h = _vp()
        _check(_lib.cgtp_norm_create(irreps.encode(), self.groups, _ACT[activation], self.eps, self.dtype_code,
                                     ctypes.byref(h)), "cgtp_norm_create")
        self._own(h, "cgtp_norm_destroy")
        v = [_i64() for _ in range(4)]
        _check(_lib.cgtp_norm_query(h, *[ctypes.byref(a) for a in v]), "cgtp_norm_query")
        self.dim, self.channels, self.biases, self.num_groups = (a.value for a in v)

    @property
    def torch_dtype(self):
        return _torch_dtype(self.dtype_code)

    def workspace_size(self, samples):
        n = _size()
        _check(_lib.cgtp_norm_workspace_size(self._h, samples._h, ctypes.byref(n)), "cgtp_norm_workspace_size")
        return n.value

    def _affine(self, weight, bias):
        if weight is not None:
            _need(weight, (self.channels,), self.torch_dtype, "weight")
        if bias is not None:
            _need(bias, (self.biases,), self.torch_dtype, "bias")

    def forward(self, samples, x, weight=None, bias=None, out=None, stats=None, ws=None):
        """(y, stats): the normalised rows and the [S, num_groups, 2] means and
        reciprocal deviations that the backward takes."""
        torch = _torch()
        dt = self.torch_dtype
        _need(x, (samples.rows, self.dim), dt, "x")
        self._affine(weight, bias)
        if out is None:
            out = torch.empty_like(x)
        _need(out, (samples.rows, self.dim), dt, "out")
        shape = (samples.S, self.num_groups, 2)
        if stats is None:
            stats = torch.empty(shape, dtype=_acc_dtype(self.dtype_code), device=x.device)
        _need(stats, shape, _acc_dtype(self.dtype_code), "stats")
        ws, nws = _workspace(ws, self.workspace_size(samples), x.device)
        _check(_lib.cgtp_norm_forward(self._h, samples._h, _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), _ptr(stats),
                                      _ptr(ws), nws, _stream(x)), "cgtp_norm_forward")
        return out, stats

    def backward(self, samples, x, weight, bias, stats, grad_y, need=(True, True, True), out=(None, None, None),
                 ws=None):
        """(grad_x, grad_weight, grad_bias)."""
        torch = _torch()
        dt = self.torch_dtype
        _need(x, (samples.rows, self.dim), dt, "x")
        _need(grad_y, (samples.rows, self.dim), dt, "grad_y")
        _need(stats, (samples.S, self.num_groups, 2), _acc_dtype(self.dtype_code), "stats")
        self._affine(weight, bias)
        shapes = [(samples.rows, self.dim), (self.channels,), (self.biases,)]
        res = []
        for k in range(3):
            if not need[k]:
                res.append(None)
                continue
            t = out[k] if out[k] is not None else torch.empty(shapes[k], dtype=dt, device=x.device)
            res.append(_need(t, shapes[k], dt, "grad"))
        ws, nws = _workspace(ws, self.workspace_size(samples), x.device)
        _check(_lib.cgtp_norm_backward(self._h, samples._h, _ptr(x), _ptr(weight), _ptr(bias), _ptr(stats),
                                       _ptr(grad_y), _ptr(res[0]), _ptr(res[1]), _ptr(res[2]), _ptr(ws), nws,
                                       _stream(x)), "cgtp_norm_backward")
        return tuple(res)


class Dropout(_Handle):
    """Dropout of irreps rows from a counter-based generator, one draw for the
    2l+1 components of a channel (cgtp_dropout_create)."""

    def __init__(self, irreps, dtype="f32"):
        self.irreps = irreps
        self.dtype_code = _DT[dtype]
        h = _vp()
        _check(_lib.cgtp_dropout_create(irreps.encode(), self.dtype_code, ctypes.byref(h)), "cgtp_dropout_create")
        self._own(h, "cgtp_dropout_destroy")
        n = _i64()
        _check(_lib.cgtp_dropout_query(h, ctypes.byref(n)), "cgtp_dropout_query")
        self.dim = n.value

    @property
    def torch_dtype(self):
        return _torch_dtype(self.dtype_code)

    @staticmethod
    def _key(seed, offset):
        if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 32:
            raise ValueError("seed must fit 64 bits and offset 32 bits, both not negative")
        return int(seed), int(offset)

    def forward(self, x, p, seed, offset, residual=None, out=None):
        """residual + dropout(x); ``offset`` differs from call to call and layer to layer."""
        shape, dt = (x.shape[0], self.dim), self.torch_dtype
        seed, offset = self._key(seed, offset)
        _need(x, shape, dt, "x")
        if residual is not None:
            _need(residual, shape, dt, "residual")
        if out is None:
            out = _torch().empty_like(x)
        _need(out, shape, dt, "out")
        _check(_lib.cgtp_dropout_forward(self._h, x.shape[0], _ptr(x), float(p), seed, offset, _ptr(residual),
                                         _ptr(out), _stream(x)), "cgtp_dropout_forward")
        return out

    def backward(self, grad_y, p, seed, offset, out=None):
        """grad_x for the forward's p, seed and offset (the residual's gradient is grad_y)."""
        shape, dt = (grad_y.shape[0], self.dim), self.torch_dtype
        seed, offset = self._key(seed, offset)
        _need(grad_y, shape, dt, "grad_y")
        if out is None:
            out = _torch().empty_like(grad_y)
        _need(out, shape, dt, "out")
        _check(_lib.cgtp_dropout_backward(self._h, grad_y.shape[0], _ptr(grad_y), float(p), seed, offset, _ptr(out),
                                          _stream(grad_y)), "cgtp_dropout_backward")
        return out
