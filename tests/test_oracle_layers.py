"""Pins of the layer oracle (oracle/layers.py): gradients against central
differences, equivariance, the generator's published test vectors."""

import numpy as np
import pytest

from oracle import layers as ol
from oracle import wigner
from oracle.irreps import dim, parse_irreps

IRREPS, GROUPS = "4x0e+2x0o+4x1o+2x2e", 2
PTR = [0, 3, 3, 4, 9]


def rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def directional(f, args, k, seed, h=1e-6):
    """(central difference, direction) of the scalar f along a random direction of args[k]."""
    d = rand(seed, *args[k].shape)
    up = [a + h * d if i == k else a for i, a in enumerate(args)]
    dn = [a - h * d if i == k else a for i, a in enumerate(args)]
    return (f(*up) - f(*dn)) / (2 * h), d


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_norm_gradients_match_differences(name):
    x, w, b = rand(0, 9, dim(parse_irreps(IRREPS))), 1 + 0.3 * rand(1, 12), 0.3 * rand(2, 4)
    g = rand(3, *x.shape)
    f = lambda x, w, b: float((g * ol.norm_forward(IRREPS, GROUPS, PTR, x, w, b, 1e-5, name)).sum())
    grads = ol.norm_backward(IRREPS, GROUPS, PTR, x, w, b, 1e-5, name, g)
    for k in range(3):
        num, d = directional(f, (x, w, b), k, 10 + k)
        # differences of step 1e-6 in fp64: h^2 truncation and eps/h rounding, about 1e-9 of the sum
        assert abs(num - float((grads[k] * d).sum())) < 1e-6 * (1 + abs(num))


def rotate(x, irreps, seed):
    angles = wigner.random_euler(np.random.default_rng(seed))
    y = np.zeros_like(x)
    for mul, l, _, off, _, _ in ol.blocks(irreps):
        n = mul * (2 * l + 1)
        D = wigner.wigner_D_real(l, *angles)
        y[:, off:off + n] = np.einsum("ab,zbu->zau", D, x[:, off:off + n].reshape(-1, 2 * l + 1, mul)).reshape(-1, n)
    return y


def test_norm_and_attention_commute_with_rotations():
    x, w, b = rand(0, 9, dim(parse_irreps(IRREPS))), 1 + 0.3 * rand(1, 12), 0.3 * rand(2, 4)
    f = lambda x: ol.norm_forward(IRREPS, GROUPS, PTR, x, w, b, 1e-5, "silu")
    assert np.abs(f(rotate(x, IRREPS, 5)) - rotate(f(x), IRREPS, 5)).max() < 1e-10
    kvi = ol.kv_irreps(IRREPS, 2, 1)
    k, v = rand(6, 7, dim(parse_irreps(kvi))), rand(7, 7, dim(parse_irreps(kvi)))
    a = lambda x, k, v: ol.attn_forward(IRREPS, 2, 1, PTR, [0, 4, 5, 5, 7], x, k, v, None, 0.4)
    o, lse = a(x, k, v)
    o2, lse2 = a(rotate(x, IRREPS, 5), rotate(k, kvi, 5), rotate(v, kvi, 5))
    assert np.abs(o2 - rotate(o, IRREPS, 5)).max() < 1e-10
    assert np.array_equal(np.isinf(lse), np.isinf(lse2))
    assert np.abs(np.where(np.isinf(lse), 0, lse2 - lse)).max() < 1e-10


def test_attention_gradients_match_differences():
    qp, kp = [0, 3, 4, 9], [0, 4, 4, 10]
    mask = np.array([1, 0, 1, 1, 1, 1, 0, 0, 1, 1], np.uint8)
    kvi = ol.kv_irreps(IRREPS, 2, 1)
    q, k, v = rand(0, 9, dim(parse_irreps(IRREPS))), rand(1, 10, dim(parse_irreps(kvi))), rand(2, 10, dim(parse_irreps(kvi)))
    g = rand(3, *q.shape)
    f = lambda q, k, v: float((g * ol.attn_forward(IRREPS, 2, 1, qp, kp, q, k, v, mask, 0.3)[0]).sum())
    grads = ol.attn_backward(IRREPS, 2, 1, qp, kp, q, k, v, mask, 0.3, g)
    for i in range(3):
        num, d = directional(f, (q, k, v), i, 20 + i)
        assert abs(num - float((grads[i] * d).sum())) < 1e-6 * (1 + abs(num))


def test_philox_published_vectors():
    full = 0xFFFFFFFF
    assert ol.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert ol.philox([full] * 4, [full] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert ol.philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_dropout_mask_rate_and_sharing():
    keep, scale = ol.dropout_mask("32x0e+32x1o", range(100), 0.25, 12345, 7)
    assert scale == 65536.0 / 49152
    # 6400 draws at 3/4: standard deviation 0.0054; six of them
    assert abs(keep[:, :64].mean() - 0.75) < 0.033
    v = keep[:, 32:].reshape(100, 3, 32)
    assert (v == v[:, :1]).all()
