"""ctypes binding of the layers on irreps rows (include/cgtp_layers.h): group
norm with its activation, attention to a context and along sequences, dropout.

As clebsch_gordan_tensor_amd.cgtp: this module checks shapes, dtypes and
devices, allocates outputs and workspaces with torch when the caller passes
none, and forwards raw pointers and the current stream. Every computation runs
in the HIP kernels of libcgtp.so.
"""

import ctypes
import weakref

import numpy as np

from .cgtp import _DT, _check, _lib, _need, _torch, _torch_dtype, _vp, _ws_bytes, F64

_i64, _size = ctypes.c_int64, ctypes.c_size_t
_i64p, _sizep, _vpp = ctypes.POINTER(_i64), ctypes.POINTER(_size), ctypes.POINTER(_vp)
_dbl, _u64, _u32 = ctypes.c_double, ctypes.c_uint64, ctypes.c_uint32

_SIGS = {
    "cgtp_samples_create": [_i64, _i64p, _vpp],
    "cgtp_samples_destroy": [_vp],
    "cgtp_norm_create": [ctypes.c_char_p, _i64, ctypes.c_int, _dbl, ctypes.c_int, _vpp],
    "cgtp_norm_destroy": [_vp],
    "cgtp_norm_query": [_vp, _i64p, _i64p, _i64p, _i64p],
    "cgtp_norm_workspace_size": [_vp, _vp, ctypes.c_int, _sizep],
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
    "cgtp_attn_batch_create_seq": [_vp, _vp, _vp, ctypes.c_int, _i64, _vpp],
    "cgtp_attn_batch_destroy": [_vp],
    "cgtp_attn_workspace_size": [_vp, ctypes.c_int, _sizep],
    "cgtp_attn_forward": [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _dbl, _vp, _vp, _vp, _size, _vp],
    "cgtp_attn_pack": [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _size, _vp],
    "cgtp_attn_forward_packed": [_vp, _vp, _i64, _vp, _size, _dbl, _vp, _vp, _vp, _size, _vp],
    "cgtp_attn_backward": [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _dbl, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                           _size, _vp],
    "cgtp_attn_cache_create": [_vp, _i64, _i64, _i64, _vpp],
    "cgtp_attn_cache_destroy": [_vp],
    "cgtp_attn_cache_query": [_vp, _sizep, _sizep],
    "cgtp_attn_cache_share": [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _size, _vp],
    "cgtp_attn_step": [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _size, _dbl, _vp, _vp, _vp, _size, _vp],
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


_raw_stream = None


def _stream_of(t):
    """The current stream's handle on t's device (the plain number: building a
    torch Stream object costs as much as a small kernel)."""
    global _raw_stream
    if _raw_stream is None:
        torch = _torch()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
    return _raw_stream(t.get_device())


def _tensor(t, shape, dtype, name):
    """t's device pointer, after _need's checks (its own path only where one fails)."""
    if t is not None and t.is_cuda and t.shape == shape and t.dtype is dtype and t.is_contiguous():
        return t.data_ptr()
    return _need(t, shape, dtype, name).data_ptr()


def _ws(ws, nbytes, device):
    """(workspace kept alive, pointer, bytes): the caller's or a new one."""
    if ws is None:
        if nbytes == 0:
            return None, 0, 0
        ws = _torch().empty(nbytes, dtype=_torch().uint8, device=device)
        return ws, ws.data_ptr(), nbytes
    return ws, ws.data_ptr(), _ws_bytes(ws)


class _Handle:
    """An opaque handle of the library, destroyed with this object."""

    _h = None
    _dtype = None

    def _own(self, handle, destroy):
        self._h, self._destroy = handle, getattr(_lib, destroy)

    @property
    def torch_dtype(self):
        if self._dtype is None:
            self._dtype = _torch_dtype(self.dtype_code)
        return self._dtype

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
        self._acc = _acc_dtype(self.dtype_code)
        self._sized = None

    def workspace_size(self, samples, backward=False):
        # (layout last used, its two sizes): layouts repeat from call to call. One value,
        # read once: another thread may put its own there meanwhile
        sized = self._sized
        if sized is None or sized[0]() is not samples:
            n, sizes = _size(), []
            for k in range(2):
                _check(_lib.cgtp_norm_workspace_size(self._h, samples._h, k, ctypes.byref(n)),
                       "cgtp_norm_workspace_size")
                sizes.append(n.value)
            sized = self._sized = weakref.ref(samples), sizes
        return sized[1][1 if backward else 0]

    def _affine(self, weight, bias):
        dt = self.torch_dtype
        return (None if weight is None else _tensor(weight, (self.channels,), dt, "weight"),
                None if bias is None else _tensor(bias, (self.biases,), dt, "bias"))

    def forward(self, samples, x, weight=None, bias=None, out=None, stats=None, ws=None):
        """(y, stats): the normalised rows and the [S, num_groups, 2] means and
        reciprocal deviations that the backward takes."""
        torch = _torch()
        dt, shape = self.torch_dtype, (samples.rows, self.dim)
        px = _tensor(x, shape, dt, "x")
        pw, pb = self._affine(weight, bias)
        if out is None:
            out = torch.empty_like(x)
        po = _tensor(out, shape, dt, "out")
        sshape, adt = (samples.S, self.num_groups, 2), self._acc
        if stats is None:
            stats = torch.empty(sshape, dtype=adt, device=x.device)
        ps = _tensor(stats, sshape, adt, "stats")
        ws, pws, nws = _ws(ws, self.workspace_size(samples), x.device)
        _check(_lib.cgtp_norm_forward(self._h, samples._h, px, pw, pb, po, ps, pws, nws, _stream_of(x)),
               "cgtp_norm_forward")
        return out, stats

    def backward(self, samples, x, weight, bias, stats, grad_y, need=(True, True, True), out=(None, None, None),
                 ws=None):
        """(grad_x, grad_weight, grad_bias)."""
        torch = _torch()
        dt, shape = self.torch_dtype, (samples.rows, self.dim)
        px = _tensor(x, shape, dt, "x")
        pg = _tensor(grad_y, shape, dt, "grad_y")
        ps = _tensor(stats, (samples.S, self.num_groups, 2), self._acc, "stats")
        pw, pb = self._affine(weight, bias)
        shapes = (shape, (self.channels,), (self.biases,))
        res = [None if not n else torch.empty(s, dtype=dt, device=x.device) if o is None else o
               for n, s, o in zip(need, shapes, out)]
        pr = [None if r is None else _tensor(r, s, dt, "grad") for r, s in zip(res, shapes)]
        ws, pws, nws = _ws(ws, self.workspace_size(samples, backward=True), x.device)
        _check(_lib.cgtp_norm_backward(self._h, samples._h, px, pw, pb, ps, pg, pr[0], pr[1], pr[2], pws, nws,
                                       _stream_of(x)), "cgtp_norm_backward")
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

    @staticmethod
    def _key(seed, offset):
        if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 32:
            raise ValueError("seed must fit 64 bits and offset 32 bits, both not negative")
        return int(seed), int(offset)

    def forward(self, x, p, seed, offset, residual=None, out=None):
        """residual + dropout(x); ``offset`` differs from call to call and layer to layer."""
        shape, dt = (x.shape[0], self.dim), self.torch_dtype
        seed, offset = self._key(seed, offset)
        px = _tensor(x, shape, dt, "x")
        pr = None if residual is None else _tensor(residual, shape, dt, "residual")
        if out is None:
            out = _torch().empty_like(x)
        _check(_lib.cgtp_dropout_forward(self._h, shape[0], px, float(p), seed, offset, pr,
                                         _tensor(out, shape, dt, "out"), _stream_of(x)), "cgtp_dropout_forward")
        return out

    def backward(self, grad_y, p, seed, offset, out=None):
        """grad_x for the forward's p, seed and offset (the residual's gradient is grad_y)."""
        shape, dt = (grad_y.shape[0], self.dim), self.torch_dtype
        seed, offset = self._key(seed, offset)
        pg = _tensor(grad_y, shape, dt, "grad_y")
        if out is None:
            out = _torch().empty_like(grad_y)
        _check(_lib.cgtp_dropout_backward(self._h, shape[0], pg, float(p), seed, offset,
                                          _tensor(out, shape, dt, "out"), _stream_of(grad_y)), "cgtp_dropout_backward")
        return out


ATTN_FORWARD, ATTN_BACKWARD, ATTN_CONTEXT, ATTN_FORWARD_PACKED = 1, 2, 3, 4


class AttentionBatch(_Handle):
    """The work lists of one pair of sample layouts (cgtp_attn_batch_create,
    cgtp_attn_batch_create_seq); made by CrossAttention.batch, reusable for every call
    on these layouts. ``nk`` counts the shared rows too."""

    def __init__(self, attn, queries, context, causal=False, shared=0):
        shared = int(shared)
        self.attn, self.nq, self.nk = attn, queries.rows, shared + context.rows     # attn outlives the handle
        self.causal, self.shared = bool(causal), shared
        h = _vp()
        if causal or shared:
            _check(_lib.cgtp_attn_batch_create_seq(attn._h, queries._h, context._h, 1 if causal else 0, shared,
                                                   ctypes.byref(h)), "cgtp_attn_batch_create_seq")
        else:
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


class AttentionCache(_Handle):
    """Keys and values of ``slots`` sequences for CrossAttention.step
    (cgtp_attn_cache_create); made by CrossAttention.cache. ``k`` and ``v`` are
    ordinary tensors of irreps rows [slots, capacity, dim_kv], to be filled with a
    prompt's rows, copied or cut like any other. ``device`` is the current one (whose
    memory the handle's tables lie in); tensors of another are refused."""

    def __init__(self, attn, slots, capacity, shared=0, device="cuda"):
        torch = _torch()
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("a cache lies in device memory, not on %s" % device)
        self._index = torch.cuda.current_device()
        if device.index not in (None, self._index):
            raise ValueError("a cache is made on the current device (%d), not on %s" % (self._index, device))
        self.attn, self.slots, self.capacity, self.shared = attn, int(slots), int(capacity), int(shared)
        h = _vp()
        _check(_lib.cgtp_attn_cache_create(attn._h, self.slots, self.capacity, self.shared, ctypes.byref(h)),
               "cgtp_attn_cache_create")
        self._own(h, "cgtp_attn_cache_destroy")
        sizes = _size(), _size()
        _check(_lib.cgtp_attn_cache_query(h, ctypes.byref(sizes[0]), ctypes.byref(sizes[1])), "cgtp_attn_cache_query")
        self._context_bytes, self.workspace_size = sizes[0].value, sizes[1].value
        shape = (self.slots, self.capacity, attn.dim_kv)
        self.k = torch.zeros(shape, dtype=attn.torch_dtype, device=device)
        self.v = torch.zeros(shape, dtype=attn.torch_dtype, device=device)
        self._context = None

    def _here(self, **tensors):
        """All of a call's tensors have to be on the cache's device (one stream and one handle serve them)."""
        for name, t in tensors.items():
            if t is not None and t.get_device() != self._index:
                raise ValueError("%s is on %s, the cache on device %d" % (name, t.device, self._index))

    def share(self, k, v, key_mask=None):
        """Lays out the rows that all sequences see before their own (cgtp_attn_cache_share), on the
        current stream. Called again it writes the same memory: steps on other streams (and replays of
        captured ones) that read the rows before or after are ordered by the caller."""
        a = self.attn
        self._here(k=k, v=v, key_mask=key_mask, cache_k=self.k)
        pk, ldk = a._rows(k, self.shared, a.dim_kv, "k")
        pv, ldv = a._rows(v, self.shared, a.dim_kv, "v")
        mask = a._mask(key_mask, self.shared)
        if self._context is None:
            self._context = _torch().empty(max(self._context_bytes, 16), dtype=_torch().uint8, device=self.k.device)
        _check(_lib.cgtp_attn_cache_share(self._h, pk, ldk, pv, ldv, mask, self._context.data_ptr(),
                                          _ws_bytes(self._context), _stream_of(self.k)), "cgtp_attn_cache_share")


class CrossAttention(_Handle):
    """Attention of irreps rows to a context of another length, sample by sample
    (cgtp_attn_create). ``irreps`` are the queries'; the context's have
    multiplicities kv_heads / heads as large (``dim_kv`` elements a row). q, k, v
    and grad_out may be slices of wider rows (unit stride within a row). With a causal
    batch whose context is the queries' own samples it is the self attention of
    sequences; ``cache`` and ``step`` continue them token by token."""

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

    def batch(self, queries, context, causal=False, shared=0):
        """``causal``: a query sees its sample's keys up to its own place, counted from
        the end. ``shared``: the first rows of k and v, before the samples' own, are seen
        by every sample (k and v have shared + context.rows rows)."""
        return AttentionBatch(self, queries, context, causal, shared)

    def cache(self, slots, capacity, shared=0, device="cuda"):
        """Caches of ``slots`` sequences for ``step``; ``shared`` rows come before all of them."""
        return AttentionCache(self, slots, capacity, shared, device)

    def _rows(self, t, rows, dim, name):
        """(pointer, row stride) of rows with unit stride inside a row."""
        if t is None:
            raise ValueError("%s is required" % name)
        if not t.is_cuda:
            raise ValueError("%s must be a device tensor" % name)
        if t.shape != (rows, dim):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, dim)))
        if t.dtype != self.torch_dtype:
            raise ValueError("%s has dtype %s, expected %s" % (name, t.dtype, self.torch_dtype))
        if t.numel() == 0:
            return t.data_ptr(), dim                                      # (its strides mean nothing)
        step, unit = t.stride()
        ld = step if rows > 1 else dim
        if (dim > 1 and unit != 1) or ld < dim:
            raise ValueError("%s must have unit stride within its rows, which may not overlap" % name)
        return t.data_ptr(), ld

    def _mask(self, m, rows):
        if m is None:
            return None
        torch = _torch()
        if m.dtype not in (torch.bool, torch.uint8):
            raise ValueError("key_mask must be bool or uint8")
        return _tensor(m, (rows,), m.dtype, "key_mask")

    def _batch(self, batch):
        if batch.attn is not self:
            raise ValueError("the batch belongs to another CrossAttention")

    def _outputs(self, batch, q, out, lse, need_lse):
        """(out, lse or None, their pointers)"""
        torch = _torch()
        if out is None:
            out = torch.empty((batch.nq, self.dim_q), dtype=self.torch_dtype, device=q.device)
        if need_lse and lse is None:
            lse = torch.empty((batch.nq, self.heads), dtype=torch.float32, device=q.device)
        return (out, lse, _tensor(out, (batch.nq, self.dim_q), self.torch_dtype, "out"),
                None if lse is None else _tensor(lse, (batch.nq, self.heads), torch.float32, "lse"))

    def forward(self, batch, q, k, v, scale=None, key_mask=None, need_lse=False, out=None, lse=None, ws=None):
        """out, or (out, lse) with ``need_lse``; scale defaults to head_dim ** -0.5."""
        self._batch(batch)
        pq, ldq = self._rows(q, batch.nq, self.dim_q, "q")
        pk, ldk = self._rows(k, batch.nk, self.dim_kv, "k")
        pv, ldv = self._rows(v, batch.nk, self.dim_kv, "v")
        mask = self._mask(key_mask, batch.nk)
        out, lse, po, pl = self._outputs(batch, q, out, lse, need_lse)
        ws, pws, nws = _ws(ws, batch.workspace_size(ATTN_FORWARD), q.device)
        _check(_lib.cgtp_attn_forward(batch._h, pq, ldq, pk, ldk, pv, ldv, mask,
                                      self.scale if scale is None else float(scale), po, pl, pws, nws, _stream_of(q)),
               "cgtp_attn_forward")
        return (out, lse) if need_lse else out

    def pack(self, batch, k, v, key_mask=None, out=None):
        """The context laid out once for any number of forward_packed calls (a uint8 tensor)."""
        self._batch(batch)
        pk, ldk = self._rows(k, batch.nk, self.dim_kv, "k")
        pv, ldv = self._rows(v, batch.nk, self.dim_kv, "v")
        mask = self._mask(key_mask, batch.nk)
        if out is None:
            out = _torch().empty(max(batch.workspace_size(ATTN_CONTEXT), 16), dtype=_torch().uint8, device=k.device)
        _check(_lib.cgtp_attn_pack(batch._h, pk, ldk, pv, ldv, mask, out.data_ptr(), _ws_bytes(out), _stream_of(k)),
               "cgtp_attn_pack")
        return out

    def forward_packed(self, batch, q, context, scale=None, need_lse=False, out=None, lse=None, ws=None):
        """forward on a packed context (of this batch or one with the same context samples)."""
        self._batch(batch)
        pq, ldq = self._rows(q, batch.nq, self.dim_q, "q")
        out, lse, po, pl = self._outputs(batch, q, out, lse, need_lse)
        ws, pws, nws = _ws(ws, batch.workspace_size(ATTN_FORWARD_PACKED), q.device)
        _check(_lib.cgtp_attn_forward_packed(batch._h, pq, ldq, context.data_ptr(), _ws_bytes(context),
                                             self.scale if scale is None else float(scale), po, pl, pws, nws,
                                             _stream_of(q)), "cgtp_attn_forward_packed")
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
        po = _tensor(out, (batch.nq, self.dim_q), dt, "out")
        pl = _tensor(lse, (batch.nq, self.heads), torch.float32, "lse")
        shapes = ((batch.nq, self.dim_q), (batch.nk, self.dim_kv), (batch.nk, self.dim_kv))
        res = [None if not n else torch.empty(s, dtype=dt, device=q.device) if g is None else g
               for n, s, g in zip(need, shapes, grads)]
        pr = [None if r is None else _tensor(r, s, dt, "grad") for r, s in zip(res, shapes)]
        ws, pws, nws = _ws(ws, batch.workspace_size(ATTN_BACKWARD), q.device)
        _check(_lib.cgtp_attn_backward(batch._h, pq, ldq, pk, ldk, pv, ldv, mask,
                                       self.scale if scale is None else float(scale), po, pl, pg, ldg, pr[0], pr[1],
                                       pr[2], pws, nws, _stream_of(q)), "cgtp_attn_backward")
        return tuple(res)

    def step(self, cache, q, k, v, lengths, scale=None, need_lse=False, out=None, lse=None, ws=None):
        """out, or (out, lse): one token of every slot, put at place lengths[s] of the caches
        and attending to the shared rows and its slot's places 0 .. lengths[s]
        (cgtp_attn_step). ``lengths`` (int32, on the device) is not changed; a slot whose
        length is not in 0 .. capacity - 1 takes no part."""
        torch = _torch()
        if cache.attn is not self:
            raise ValueError("the cache belongs to another CrossAttention")
        n, dt = cache.slots, self.torch_dtype
        if cache.shared and cache._context is None:
            raise ValueError("the cache's shared rows have not been laid out (share)")
        cache._here(q=q, k=k, v=v, lengths=lengths, out=out, lse=lse, ws=ws, cache_k=cache.k, cache_v=cache.v)
        pq, ldq = self._rows(q, n, self.dim_q, "q")
        pk, ldk = self._rows(k, n, self.dim_kv, "k")
        pv, ldv = self._rows(v, n, self.dim_kv, "v")
        shape = (n, cache.capacity, self.dim_kv)
        ck, cv = _tensor(cache.k, shape, dt, "cache.k"), _tensor(cache.v, shape, dt, "cache.v")
        pn = _tensor(lengths, (n,), torch.int32, "lengths")
        if out is None:
            out = torch.empty((n, self.dim_q), dtype=dt, device=q.device)
        if need_lse and lse is None:
            lse = torch.empty((n, self.heads), dtype=torch.float32, device=q.device)
        po = _tensor(out, (n, self.dim_q), dt, "out")
        pl = None if lse is None else _tensor(lse, (n, self.heads), torch.float32, "lse")
        ws, pws, nws = _ws(ws, cache.workspace_size, q.device)
        shared = (None, 0) if not cache.shared else (cache._context.data_ptr(), _ws_bytes(cache._context))
        _check(_lib.cgtp_attn_step(cache._h, pq, ldq, pk, ldk, pv, ldv, ck, cv, pn, shared[0], shared[1],
                                   self.scale if scale is None else float(scale), po, pl, pws, nws, _stream_of(q)),
               "cgtp_attn_step")
        return (out, lse) if need_lse else out
