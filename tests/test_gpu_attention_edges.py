"""GPU cross attention at the edges of its range: split contexts with parts that
the mask empties, NaN in queries, values far from one, limits of its arguments."""

import numpy as np
import pytest

from oracle import layers as ol
from tests.gpu_util import TOL, dev, host, rel_err
from tests.test_gpu_attention import inputs, ptr_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [3, 40, 300])                 # few rows; 32 rows a wave; 64 rows a wave (bf16)
def test_split_context_whose_last_parts_are_masked(dtype, nq):
    """Scores near -196 against the first 200 of 2500 keys, the rest masked: a part
    without a key must not count as one of score 0.

    A score is a sum of 32 products of size 6: rounding leaves at most 32 * 2^-24 * 196
    = 3.7e-4 of it, twice that of a weight and of its share in the result, so 2e-3 of
    the largest value covers fp32; bf16 adds its own rounding."""
    irreps, nk, seen = "32x0e", 2500, 200
    attn = layers.CrossAttention(irreps, 1, dtype=dtype)
    rng = np.random.default_rng(31)
    base = 14.0 / np.sqrt(32)
    q = dev(-base + 0.1 * rng.standard_normal((nq + 2, 32)), dtype)
    k = dev(base + 0.1 * rng.standard_normal((nk + 900, 32)), dtype)
    v, g = dev(rng.standard_normal((nk + 900, 32)), dtype), dev(rng.standard_normal((nq + 2, 32)), dtype)
    mask = torch.zeros(nk + 900, dtype=torch.bool, device="cuda")
    mask[:seen] = True                                       # the second sample keeps none of its 900 keys
    qp, kp = ptr_of([nq, 2]), ptr_of([nk, 900])
    b = attn.batch(layers.Samples(qp), layers.Samples(kp))
    assert b.workspace_size(layers.ATTN_FORWARD_PACKED) > 0  # the contexts are split
    out, lse = attn.forward(b, q, k, v, scale=1.0, key_mask=mask, need_lse=True)
    dv = attn.backward(b, q, k, v, out, lse, g, scale=1.0, key_mask=mask)[2]
    torch.cuda.synchronize()
    args = (irreps, 1, 1, qp, kp, host(q), host(k), host(v), mask.cpu().numpy(), 1.0)
    ro, rl = ol.attn_forward(*args)
    rdv = ol.attn_backward(*args, host(g))[2]
    tol = 2e-3 if dtype == "f32" else TOL[dtype]
    assert np.array_equal(np.isinf(host(lse)), np.isinf(rl))
    assert np.abs(host(lse)[:nq] - rl[:nq]).max() <= 1e-3
    assert rel_err(host(out), ro) <= tol and rel_err(host(dv), rdv) <= tol
    assert torch.all(out[nq:] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,heads", [("32x0e+16x1o", 4), ("48x0e+48x1o", 1)])  # both gradients in one pass; in two
@pytest.mark.parametrize("where", ["query", "key"])
def test_masked_keys_have_no_gradient_beside_nan(where, irreps, heads, dtype):
    nq, nk = [40, 300], [90, 700]
    attn = layers.CrossAttention(irreps, heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, heads, nq, nk, dtype)
    mask = torch.from_numpy(np.random.default_rng(6).random(sum(nk)) < 0.6).cuda()
    mask[3] = True
    (q if where == "query" else k)[3] = float("nan")
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))
    out, lse = attn.forward(b, q, k, v, key_mask=mask, need_lse=True)
    _, dk, dv = attn.backward(b, q, k, v, out, lse, g, key_mask=mask)
    assert torch.isnan(out[3]).all() and torch.isnan(dk[3]).all()
    assert torch.all(dk[~mask] == 0) and torch.all(dv[~mask] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [[40, 3, 70], [1, 1, 1], [5, 300, 9]])
@pytest.mark.parametrize("where", ["query", "key"])
def test_nan_reaches_the_gradients(where, nq, dtype):
    """A NaN in a query with keys is in its own gradient and in those of all keys that it
    sees; one in a visible key is in every gradient of its sample; none is in another
    sample's."""
    irreps, heads, kv_heads, nk = "32x0e+16x1o", 4, 2, [90, 45, 64]
    qp, kp = ptr_of(nq), ptr_of(nk)
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, kv_heads, nq, nk, dtype)
    b = attn.batch(layers.Samples(qp), layers.Samples(kp))
    ref = ol.attn_backward(irreps, heads, kv_heads, qp, kp, host(q), host(k), host(v), None, attn.scale, host(g))
    keys = slice(kp[1], kp[2])
    if where == "query":
        q[qp[1]] = float("nan")
        rows = slice(qp[1], qp[1] + 1)
    else:
        k[kp[1] + 7] = float("nan")
        rows = slice(qp[1], qp[2])
    out, lse = attn.forward(b, q, k, v, need_lse=True)
    grads = [host(t) for t in attn.backward(b, q, k, v, out, lse, g)]
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    # all else as without it, judged against the largest gradient of its kind
    for got, want, bad in zip(grads, ref, (rows, keys, keys)):
        assert np.isnan(got[bad]).all()
        rest = np.delete(got, bad, 0)
        scale = max(np.abs(want).max(), 0.1 * max(np.abs(r).max() for r in ref))
        assert np.abs(rest - np.delete(want, bad, 0)).max() <= TOL[dtype] * scale


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [[40, 3, 70], [1, 1, 1], [5, 300, 9]])
def test_nan_queries_without_a_key(dtype, nq):
    """Rows that see no key are 0 with lse -inf whatever they hold, and reach no gradient."""
    irreps, heads, kv_heads, nk = "32x0e+16x1o", 4, 2, [90, 45, 64]
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, kv_heads, nq, nk, dtype)
    mask = torch.from_numpy(np.random.default_rng(5).random(sum(nk)) < 0.6).cuda()
    mask[0] = mask[-1] = True
    mask[90:135] = False                                     # the second sample has no key left
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))

    def step(q):
        out, lse = attn.forward(b, q, k, v, key_mask=mask, need_lse=True)
        packed = attn.forward_packed(b, q, attn.pack(b, k, v, key_mask=mask))
        return (out, packed, lse) + attn.backward(b, q, k, v, out, lse, g, key_mask=mask)

    want = step(q)
    rows = slice(nq[0], nq[0] + nq[1])
    assert torch.all(want[0][rows] == 0) and torch.all(want[2][rows] == -float("inf"))
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[rows] = bad
        assert all(torch.equal(x, y) for x, y in zip(step(q2), want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [3, 40, 300])
@pytest.mark.parametrize("sign,size", [(1, 2.0 ** 105), (-1, 2.0 ** 105), (1, 2.0 ** -60), (-1, 2.0 ** -60)])
def test_values_far_from_one(dtype, nq, sign, size):
    """Scores of +-16 (2^+-23 as weights without a reference) with values whose products
    with such weights leave fp32: the result is a mean of the values all the same.

    A score of 16 from 32 products carries at most 32 * 2^-24 * 16 = 3e-5; its weight
    and the result twice that at most."""
    irreps, nk = "32x0e", 200
    attn = layers.CrossAttention(irreps, 1, dtype=dtype)
    rng = np.random.default_rng(41)
    base = 4.0 / np.sqrt(32)
    q = dev(sign * base + 0.02 * rng.standard_normal((nq, 32)), dtype)
    k = dev(base + 0.02 * rng.standard_normal((nk, 32)), dtype)
    v = dev(size * (1 + rng.random((nk, 32))), dtype)
    b = attn.batch(layers.Samples([0, nq]), layers.Samples([0, nk]))
    out, lse = attn.forward(b, q, k, v, scale=1.0, need_lse=True)
    torch.cuda.synchronize()
    ro, rl = ol.attn_forward(irreps, 1, 1, [0, nq], [0, nk], host(q), host(k), host(v), None, 1.0)
    assert rel_err(host(out), ro) <= (1e-4 if dtype == "f32" else TOL[dtype])
    assert np.abs(host(lse) - rl).max() <= 1e-4


def test_scale_beyond_fp32_is_refused():
    # finite in 64 bits, infinite in the kernels' 32 (times log2 e): 0 * inf would be NaN
    attn = layers.CrossAttention("16x0e", 2)
    b = attn.batch(layers.Samples([0, 3]), layers.Samples([0, 5]))
    q, k = torch.zeros((3, 16), device="cuda"), torch.ones((5, 16), device="cuda")
    out, lse = attn.forward(b, q, k, k, scale=2e38, need_lse=True)
    assert torch.all(out == 1)
    ctx = attn.pack(b, k, k)
    for scale in (1e39, -3e38, float("nan")):
        for bad in (lambda: attn.forward(b, q, k, k, scale=scale),
                    lambda: attn.forward_packed(b, q, ctx, scale=scale),
                    lambda: attn.backward(b, q, k, k, out, lse, q, scale=scale)):
            with pytest.raises(cgtp.CgtpError) as e:
                bad()
            assert e.value.status == 1


def test_more_tiles_than_one_launch_takes_are_refused():
    attn = layers.CrossAttention("256x0e", 256, dtype="bf16")
    one, many = (layers.Samples(np.arange(n + 1)) for n in (1000, 65_600))       # 256 tiles a sample of one row
    attn.batch(one, one)
    with pytest.raises(cgtp.CgtpError) as e:
        attn.batch(many, many)
    assert e.value.status == 3


def test_strides_of_tensors_without_elements_are_not_judged():
    attn = layers.CrossAttention("16x0e+8x1o", 4)
    b = attn.batch(layers.Samples([0, 0]), layers.Samples([0, 0]))
    none = torch.empty((0, attn.dim_q), device="cuda").as_strided((0, attn.dim_q), (0, 0))   # as NumPy's come
    out, lse = attn.forward(b, none, none, none, need_lse=True)
    grads = attn.backward(b, none, none, none, out, lse, none)
    assert all(t.shape == none.shape for t in (out, *grads))
    attn.forward_packed(b, none, attn.pack(b, none, none))
