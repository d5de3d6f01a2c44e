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
    "cgtp_attn_create": [ctypes.c_char_p, _i64, _i64, ctypes.c_int, _vpp],
    "cgtp_attn_destroy": [_vp],
    "cgtp_attn_query": [_vp, _i64p, _i64p, _i64p],
    "cgtp_attn_batch_create": [_vp, _vp, _vp, _vpp],
    "cgtp_attn_batch_destroy": [_vp],
    "cgtp_attn_workspace_size": [_vp, ctypes.c_int, _sizep],
    "cgtp_attn_forward": [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _dbl, _vp, _vp, _vp, _size, _vp],
    "cgtp_attn_pack": [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _size, _vp],
    "cgtp_attn_forward_packed": [_vp, _vp, _i64, _vp, _size, _dbl, _vp, _vp, _vp, _size, _vp],
    "cgtp_attn_backward": [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _dbl, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                           _size, _vp],
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


ATTN_FORWARD, ATTN_BACKWARD, ATTN_CONTEXT, ATTN_FORWARD_PACKED = 1, 2, 3, 4


class AttentionBatch(_Handle):
    """The work lists of one pair of sample layouts (cgtp_attn_batch_create);
    made by CrossAttention.batch, reusable for every call on these layouts."""

    def __init__(self, attn, queries, context):
        self.attn, self.nq, self.nk = attn, queries.rows, context.rows     # attn outlives the handle
        h = _vp()
        _check(_lib.cgtp_attn_batch_create(attn._h, queries._h, context._h, ctypes.byref(h)),
               "cgtp_attn_batch_create")
        self._own(h, "cgtp_attn_batch_destroy")
        self._sizes = {}

    def workspace_size(self, op):
        if op not in self._sizes:
            n = _size()
            _check(_lib.cgtp_attn_workspace_size(self._h, op, ctypes.byref(n)), "cgtp_attn_workspace_size")
            self._sizes[op] = n.value
        return self._sizes[op]


class CrossAttention(_Handle):
    """Attention of irreps rows to a context of another length, sample by sample
    (cgtp_attn_create). ``irreps`` are the queries'; the context's have
    multiplicities kv_heads / heads as large (``dim_kv`` elements a row). q, k, v
    and grad_out may be slices of wider rows (unit stride within a row)."""

    def __init__(self, irreps, heads, kv_heads=None, dtype="f32"):
        self.irreps, self.heads = irreps, int(heads)
        self.kv_heads = self.heads if kv_heads is None else int(kv_heads)
        self.dtype_code = _DT[dtype]
        h = _vp()
        _check(_lib.cgtp_attn_create(irreps.encode(), self.heads, self.kv_heads, self.dtype_code, ctypes.byref(h)),
               "cgtp_attn_create")
        self._own(h, "cgtp_attn_destroy")
        v = [_i64() for _ in range(3)]
        _check(_lib.cgtp_attn_query(h, *[ctypes.byref(a) for a in v]), "cgtp_attn_query")
        self.dim_q, self.dim_kv, self.head_dim = (a.value for a in v)
        self.scale = self.head_dim ** -0.5

    @property
    def torch_dtype(self):
        return _torch_dtype(self.dtype_code)

    def batch(self, queries, context):
        return AttentionBatch(self, queries, context)

    def _rows(self, t, rows, dim, name):
        """(pointer, row stride) of rows with unit stride inside a row."""
        if t is None:
            raise ValueError("%s is required" % name)
        if not t.is_cuda:
            raise ValueError("%s must be a device tensor" % name)
        if tuple(t.shape) != (rows, dim):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, dim)))
        if t.dtype != self.torch_dtype:
            raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, self.torch_dtype))
        ld = t.stride(0) if rows > 1 else dim
        if (dim > 1 and t.stride(1) != 1) or ld < dim:
            raise ValueError("%s must have unit stride within its rows, which may not overlap" % name)
        return _ptr(t), ld

    def _mask(self, m, rows):
        if m is None:
            return _vp(0)
        torch = _torch()
        if m.dtype not in (torch.bool, torch.uint8):
            raise ValueError("key_mask must be bool or uint8")
        return _ptr(_need(m, (rows,), m.dtype, "key_mask"))

    def _batch(self, batch):
        if batch.attn is not self:
            raise ValueError("the batch belongs to another CrossAttention")

    def _outputs(self, batch, q, out, lse, need_lse):
        torch = _torch()
        if out is None:
            out = torch.empty((batch.nq, self.dim_q), dtype=self.torch_dtype, device=q.device)
        _need(out, (batch.nq, self.dim_q), self.torch_dtype, "out")
        if need_lse and lse is None:
            lse = torch.empty((batch.nq, self.heads), dtype=torch.float32, device=q.device)
        if lse is not None:
            _need(lse, (batch.nq, self.heads), torch.float32, "lse")
        return out, lse

    def forward(self, batch, q, k, v, scale=None, key_mask=None, need_lse=False, out=None, lse=None, ws=None):
        """out, or (out, lse) with ``need_lse``; scale defaults to head_dim ** -0.5."""
        self._batch(batch)
        pq, ldq = self._rows(q, batch.nq, self.dim_q, "q")
        pk, ldk = self._rows(k, batch.nk, self.dim_kv, "k")
        pv, ldv = self._rows(v, batch.nk, self.dim_kv, "v")
        mask = self._mask(key_mask, batch.nk)
        out, lse = self._outputs(batch, q, out, lse, need_lse)
        ws, nws = _workspace(ws, batch.workspace_size(ATTN_FORWARD), q.device)
        _check(_lib.cgtp_attn_forward(batch._h, pq, ldq, pk, ldk, pv, ldv, mask,
                                      self.scale if scale is None else float(scale), _ptr(out), _ptr(lse), _ptr(ws),
                                      nws, _stream(q)), "cgtp_attn_forward")
        return (out, lse) if need_lse else out

    def pack(self, batch, k, v, key_mask=None, out=None):
        """The context laid out once for any number of forward_packed calls (a uint8 tensor)."""
        self._batch(batch)
        pk, ldk = self._rows(k, batch.nk, self.dim_kv, "k")
        pv, ldv = self._rows(v, batch.nk, self.dim_kv, "v")
        mask = self._mask(key_mask, batch.nk)
        out, n = _workspace(out, batch.workspace_size(ATTN_CONTEXT), k.device)
        _check(_lib.cgtp_attn_pack(batch._h, pk, ldk, pv, ldv, mask, _ptr(out), n, _stream(k)), "cgtp_attn_pack")
        return out

    def forward_packed(self, batch, q, context, scale=None, need_lse=False, out=None, lse=None, ws=None):
        """forward on a packed context (of this batch or one with the same context samples)."""
        self._batch(batch)
        pq, ldq = self._rows(q, batch.nq, self.dim_q, "q")
        out, lse = self._outputs(batch, q, out, lse, need_lse)
        ws, nws = _workspace(ws, batch.workspace_size(ATTN_FORWARD_PACKED), q.device)
        _check(_lib.cgtp_attn_forward_packed(batch._h, pq, ldq, _ptr(context), _ws_bytes(context),
                                             self.scale if scale is None else float(scale), _ptr(out), _ptr(lse),
                                             _ptr(ws), nws, _stream(q)), "cgtp_attn_forward_packed")
        return (out, lse) if need_lse else out

    def backward(self, batch, q, k, v, out, lse, grad_out, scale=None, key_mask=None, need=(True, True, True),
                 grads=(None, None, None), ws=None):
        """(grad_q, grad_k, grad_v) from the forward's out and lse."""
        torch = _torch()
        self._batch(batch)
        dt = self.torch_dtype
        pq, ldq = self._rows(q, batch.nq, self.dim_q, "q")
        pk, ldk = self._rows(k, batch.nk, self.dim_kv, "k")
        pv, ldv = self._rows(v, batch.nk, self.dim_kv, "v")
        pg, ldg = self._rows(grad_out, batch.nq, self.dim_q, "grad_out")
        mask = self._mask(key_mask, batch.nk)
        _need(out, (batch.nq, self.dim_q), dt, "out")
        _need(lse, (batch.nq, self.heads), torch.float32, "lse")
        shapes = [(batch.nq, self.dim_q), (batch.nk, self.dim_kv), (batch.nk, self.dim_kv)]
        res = []
        for i in range(3):
            if not need[i]:
                res.append(None)
                continue
            t = grads[i] if grads[i] is not None else torch.empty(shapes[i], dtype=dt, device=q.device)
            res.append(_need(t, shapes[i], dt, "grad"))
        ws, nws = _workspace(ws, batch.workspace_size(ATTN_BACKWARD), q.device)
        _check(_lib.cgtp_attn_backward(batch._h, pq, ldq, pk, ldk, pv, ldv, mask,
                                       self.scale if scale is None else float(scale), _ptr(out), _ptr(lse), pg, ldg,
                                       *[_ptr(t) for t in res], _ptr(ws), nws, _stream(q)), "cgtp_attn_backward")
        return tuple(res)
