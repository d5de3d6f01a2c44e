"""Host-side checks of the layer entry points (CPU only): the header's functions
are exported and bound, malformed requests return the documented codes."""

import ctypes
import os
import re

import numpy as np
import pytest

cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "cgtp_layers.h")
INVALID, PARSE, UNSUPPORTED, INDEX = 1, 2, 3, 4


def test_every_declared_symbol_is_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(cgtp_[a-z_]+)\s*\(", text)))
    assert names == sorted(layers.EXPORTED)
    assert all(hasattr(cgtp._lib, n) for n in names)


def status_of(fn):
    with pytest.raises(cgtp.CgtpError) as e:
        fn()
    return e.value.status


def test_create_errors():
    assert status_of(lambda: layers.Samples([1, 2])) == INDEX
    assert status_of(lambda: layers.Samples([0, 3, 2])) == INDEX
    assert status_of(lambda: layers.Samples([0, 1 << 31])) == UNSUPPORTED
    with pytest.raises(ValueError):
        layers.Samples([])
    with pytest.raises(ValueError):
        layers.Samples(np.array([0.0, 1.0]))
    assert status_of(lambda: layers.GroupNorm("8x0q", 2)) == PARSE
    assert status_of(lambda: layers.GroupNorm("8x0e+6x1o", 4)) == UNSUPPORTED
    assert status_of(lambda: layers.GroupNorm("8x5o", 2)) == UNSUPPORTED
    assert status_of(lambda: layers.GroupNorm("", 1)) == UNSUPPORTED
    assert status_of(lambda: layers.GroupNorm("8x0e", 0)) == INVALID
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert status_of(lambda: layers.GroupNorm("8x0e", 2, eps=eps)) == INVALID
    assert status_of(lambda: layers.Dropout("3x")) == PARSE
    assert status_of(lambda: layers.Dropout("3x5e")) == UNSUPPORTED
    assert status_of(lambda: layers.Dropout("300000x0e")) == UNSUPPORTED
    assert status_of(lambda: layers.CrossAttention("8x0e+6x1o", 4)) == UNSUPPORTED
    assert status_of(lambda: layers.CrossAttention("8x0e", 4, kv_heads=3)) == INVALID
    assert status_of(lambda: layers.CrossAttention("8x0e", 0)) == INVALID
    assert status_of(lambda: layers.CrossAttention("8x0e", 4, kv_heads=8)) == INVALID
    assert status_of(lambda: layers.CrossAttention("257x0e", 1)) == UNSUPPORTED
    assert status_of(lambda: layers.CrossAttention("8x0e", 4, dtype="f64")) == UNSUPPORTED


def test_null_arguments():
    lib, n = cgtp._lib, None
    sz = ctypes.c_size_t()
    assert lib.cgtp_samples_create(1, n, n) == INVALID
    assert lib.cgtp_norm_create(n, 1, 0, 1e-5, 0, n) == INVALID
    assert lib.cgtp_norm_forward(n, n, n, n, n, n, n, n, 0, n) == INVALID
    assert lib.cgtp_norm_backward(*([n] * 11), 0, n) == INVALID
    assert lib.cgtp_norm_workspace_size(n, n, 0, ctypes.byref(sz)) == INVALID
    assert lib.cgtp_dropout_forward(n, 1, n, 0.1, 0, 0, n, n, n) == INVALID
    assert lib.cgtp_attn_create(n, 1, 1, 0, n) == INVALID
    assert lib.cgtp_attn_batch_create(n, n, n, n) == INVALID
    assert lib.cgtp_attn_workspace_size(n, 1, ctypes.byref(sz)) == INVALID
    assert lib.cgtp_attn_forward(n, n, 0, n, 0, n, 0, n, 1.0, n, n, n, 0, n) == INVALID
    assert lib.cgtp_attn_pack(n, n, 0, n, 0, n, n, 0, n) == INVALID
    assert lib.cgtp_attn_forward_packed(n, n, 0, n, 0, 1.0, n, n, n, 0, n) == INVALID
    assert lib.cgtp_attn_backward(n, n, 0, n, 0, n, 0, n, 1.0, n, n, n, 0, n, n, n, n, 0, n) == INVALID
    for f in ("samples", "norm", "dropout", "attn", "attn_batch"):
        assert getattr(lib, "cgtp_%s_destroy" % f)(n) == 0
