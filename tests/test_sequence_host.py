"""Host-side checks of the attention along sequences (CPU only): malformed requests
return the documented codes; the oracle agrees with attention written from its definition."""

import ctypes

import numpy as np
import pytest

from oracle import layers as ol
from oracle.irreps import dim, parse_irreps

cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

INVALID = 1


def test_null_arguments():
    lib, n = cgtp._lib, None
    h, sz = ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.cgtp_attn_batch_create_seq(n, n, n, 1, 0, ctypes.byref(h)) == INVALID
    assert lib.cgtp_attn_batch_create_seq(n, n, n, 1, 0, n) == INVALID
    assert lib.cgtp_attn_cache_create(n, 1, 1, 0, ctypes.byref(h)) == INVALID
    assert lib.cgtp_attn_cache_create(n, 1, 1, 0, n) == INVALID
    assert lib.cgtp_attn_cache_query(n, ctypes.byref(sz), ctypes.byref(sz)) == INVALID
    assert lib.cgtp_attn_cache_share(n, n, 0, n, 0, n, n, 0, n) == INVALID
    assert lib.cgtp_attn_step(n, n, 0, n, 0, n, 0, n, n, n, n, 0, 1.0, n, n, n, 0, n) == INVALID
    assert lib.cgtp_attn_cache_destroy(n) == 0


def naive(irreps, heads, kv_heads, q, k, v, seen, scale):
    """Softmax over the seen keys, head by head and element by element."""
    out = np.zeros_like(q)
    for h in range(heads):
        qc = ol.head_columns(irreps, heads, h)
        kc = ol.head_columns(ol.kv_irreps(irreps, heads, kv_heads), kv_heads, h * kv_heads // heads)
        for i in range(len(q)):
            at = np.flatnonzero(seen[i])
            if len(at):
                w = np.exp([scale * float(q[i, qc] @ k[j, kc]) for j in at])
                out[i, qc] = sum(a * v[j, kc] for a, j in zip(w, at)) / w.sum()
    return out


@pytest.mark.parametrize("nq,nk,causal,shared", [(5, 5, True, 0), (3, 7, True, 0), (6, 2, True, 0), (4, 4, True, 3),
                                                 (4, 0, False, 3), (6, 2, True, 1), (4, 5, False, 2)])
def test_oracle_of_sequences(nq, nk, causal, shared):
    irreps, heads, kv_heads = "4x0e+2x1o", 2, 1
    rng = np.random.default_rng(0)
    q = rng.standard_normal((2 + nq, dim(parse_irreps(irreps))))
    k, v = (rng.standard_normal((shared + 3 + nk, dim(parse_irreps(ol.kv_irreps(irreps, heads, kv_heads))))) for _ in "kv")
    mask = np.ones(len(k))
    mask[-1] = 0
    seen = np.zeros((2 + nq, len(k)), bool)
    seen[:, :shared] = True
    for i in range(2):                                # a sample of 2 queries and 3 keys, then the one asked for
        seen[i, shared:shared + (3 if not causal else i + 2)] = True
    for i in range(nq):
        n = nk if not causal else max(0, i + nk - nq + 1)
        seen[2 + i, shared + 3:shared + 3 + n] = True
    seen &= mask != 0
    args = (irreps, heads, kv_heads, [0, 2, 2 + nq], [0, 3, 3 + nk], q, k, v, mask, 0.3)
    out, lse = ol.seq_forward(*args, causal, shared)
    assert np.abs(out - naive(irreps, heads, kv_heads, q, k, v, seen, 0.3)).max() <= 1e-12
    assert np.array_equal(np.isinf(lse[:, 0]), ~seen.any(1))
    g = rng.standard_normal(q.shape)
    grads = ol.seq_backward(*args, g, causal, shared)
    for i, x in enumerate((q, k, v)):
        d, h = rng.standard_normal(x.shape), 1e-6
        sides = []
        for sign in (h, -h):
            moved = [q, k, v]
            moved[i] = x + sign * d
            sides.append((ol.seq_forward(*args[:5], *moved, mask, 0.3, causal, shared)[0] * g).sum())
        assert abs((sides[0] - sides[1]) / (2 * h) - (grads[i] * d).sum()) <= 1e-7


def test_oracle_of_a_step_is_that_of_a_causal_batch():
    irreps, heads, kv_heads, shared = "4x0e+2x1o", 2, 1, 3
    rng = np.random.default_rng(1)
    q = rng.standard_normal((9, 10))
    k, v = (rng.standard_normal((shared + 9, 5)) for _ in "kv")
    want, lse = ol.seq_forward(irreps, heads, kv_heads, [0, 9], [0, 9], q, k, v, None, 0.3, True, shared)
    kc, vc = np.full((1, 8, 5), np.nan), np.full((1, 8, 5), np.nan)
    for n in range(9):
        at = slice(shared + n, shared + n + 1)
        out, l, kc, vc = ol.cache_step(irreps, heads, kv_heads, q[n:n + 1], k[at], v[at], kc, vc, [n], 0.3,
                                       (k[:shared], v[:shared], None))
        if n < 8:
            assert np.abs(out - want[n]).max() <= 1e-12 and np.abs(l - lse[n]).max() <= 1e-12
        else:
            assert not out.any() and np.isinf(l).all()
