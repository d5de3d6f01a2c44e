"""GPU cross attention against the fp64 oracle: ragged, empty and single-key
samples, lengths from one token to thousands, grouped heads, odd channel counts
and head sizes up to 256, masks that leave rows empty, infinities and NaN in
masked places, strided rows, split contexts, the packed form; gradients also
against differences; streams, graph capture, refusals."""

import numpy as np
import pytest

from oracle import layers as ol
from oracle.irreps import dim, parse_irreps
from tests.gpu_util import TOL, dev, host, rel_err, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

# (irreps, heads, kv heads, query lengths, context lengths)
CASES = [
    ("32x0e+32x1o+32x2e", 4, 4, [9, 21, 0, 1], [0, 60, 5, 33]),
    ("10x0e+6x1o", 2, 1, [3, 70], [1, 65]),                         # head of 14 elements, element-wise rows
    ("35x0e+21x1o+7x2e", 7, 1, [40, 1], [31, 130]),                 # 7 heads share a context head
    ("64x0e", 2, 2, [129, 32], [64, 32]),                           # exact tiles
    ("128x0e+128x1o", 4, 4, [150], [300]),                          # head of 128
    ("128x0e+128x1o+128x2e", 8, 4, [50, 140], [200, 90]),           # 144, padded to 160
    ("96x0e+96x1o+24x2e", 6, 3, [65], [97]),                        # 84
    ("24x0e+24x1o+24x2e+24x3o", 2, 1, [33], [50]),                  # 192
    ("14x0e+14x1o+14x2e+14x3o", 1, 1, [40], [70]),                  # 224
    ("128x0e+128x1o+128x2e+128x3o", 8, 8, [70], [40]),              # 256
    ("128x0e+128x1o+128x2e+128x3o", 16, 4, [1, 1, 1], [700, 1, 2500]),   # single tokens, split
    ("16x0e", 4, 2, [2, 700], [2300, 40]),                          # both kernels, both splits
    ("8x0e", 1, 1, [1], [1]),
]


def inputs(irreps, heads, kv_heads, nq, nk, dtype, seed=0):
    rng = np.random.default_rng(seed)
    d = dim(parse_irreps(irreps))
    dk = dim(parse_irreps(ol.kv_irreps(irreps, heads, kv_heads)))
    return [dev(rng.standard_normal(s), dtype) for s in ((sum(nq), d), (sum(nk), dk), (sum(nk), dk), (sum(nq), d))]


def ptr_of(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def compare(attn, irreps, heads, kv_heads, nq, nk, dtype, q, k, v, g, mask=None, refs=None):
    qp, kp = ptr_of(nq), ptr_of(nk)
    batch = attn.batch(layers.Samples(qp), layers.Samples(kp))
    out, lse = attn.forward(batch, q, k, v, key_mask=mask, need_lse=True)
    grads = attn.backward(batch, q, k, v, out, lse, g, key_mask=mask)
    packed = attn.forward_packed(batch, q, attn.pack(batch, k, v, key_mask=mask))
    torch.cuda.synchronize()
    hm = None if mask is None else mask.cpu().numpy()
    hq, hk, hv, hg = refs or (host(q), host(k), host(v), host(g))
    ro, rl = ol.attn_forward(irreps, heads, kv_heads, qp, kp, hq, hk, hv, hm, attn.scale)
    rg = ol.attn_backward(irreps, heads, kv_heads, qp, kp, hq, hk, hv, hm, attn.scale, hg)
    assert torch.equal(packed, out)
    assert rel_err(host(out), ro) <= TOL[dtype]
    gl = host(lse)
    assert np.array_equal(np.isinf(gl), np.isinf(rl))
    fin = np.isfinite(rl)
    # lse: fp32 sums and logarithms of scores of size 10 at most; bf16 only rounds the inputs, which both sides share
    assert fin.sum() == 0 or np.abs(gl[fin] - rl[fin]).max() <= 2e-5
    for name, a, b in zip(("grad_q", "grad_k", "grad_v"), grads, rg):
        assert np.isfinite(host(a)).all()
        # a gradient that is zero in exact arithmetic (one key) is judged against the others' size
        scale = max(np.abs(b).max() if b.size else 0.0, 0.1 * max(np.abs(r).max() if r.size else 0.0 for r in rg))
        err = np.abs(host(a) - b).max() if b.size else 0.0
        assert err <= TOL[dtype] * scale, "%s: %.3e of %.3e" % (name, err, scale)
    return (out, lse) + grads


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,heads,kv_heads,nq,nk", CASES)
def test_attention(irreps, heads, kv_heads, nq, nk, dtype):
    print("attention", irreps, heads, kv_heads, nq, nk, dtype, flush=True)
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, kv_heads, nq, nk, dtype)
    a = compare(attn, irreps, heads, kv_heads, nq, nk, dtype, q, k, v, g)
    b = compare(attn, irreps, heads, kv_heads, nq, nk, dtype, q, k, v, g)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq", [[40, 3, 70], [1, 1, 1]])
def test_masks_with_nan_and_inf_in_masked_places(dtype, nq):
    irreps, heads, kv_heads, nk = "32x0e+16x1o", 4, 2, [90, 33, 64]
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, kv_heads, nq, nk, dtype)
    mask = torch.from_numpy(np.random.default_rng(5).random(sum(nk)) < 0.6).cuda()
    mask[90:123] = False                              # the second sample has no key left
    mask[-1], mask[0] = True, False
    refs = [host(t) for t in (q, k, v, g)]
    for t, bad in ((k, float("nan")), (v, float("inf"))):
        t[~mask] = bad
    refs[1][~mask.cpu().numpy()] = 0
    refs[2][~mask.cpu().numpy()] = 0
    lo, hi = nq[0], nq[0] + nq[1]
    g[lo:hi] = float("nan")                           # gradients of rows that saw nothing do not spread
    refs[3][lo:hi] = 0
    for m in (mask, mask.to(torch.uint8) * 3):
        out, lse, dq, dk, dv = compare(attn, irreps, heads, kv_heads, nq, nk, dtype, q, k, v, g, mask=m, refs=refs)
        assert torch.all(out[lo:hi] == 0) and torch.all(dq[lo:hi] == 0) and torch.all(torch.isinf(lse[lo:hi]))
        assert torch.all(dk[~mask] == 0) and torch.all(dv[~mask] == 0)


@pytest.mark.parametrize("dtype,rows,heads,irreps", [("f32", 50, 2, "32x0e"), ("bf16", 300, 2, "32x0e"),
                                                     ("bf16", 300, 1, "32x0e+32x1o"), ("bf16", 90, 1, "160x0e"),
                                                     ("bf16", 1, 2, "32x0e")])
def test_large_scores_do_not_overflow(dtype, rows, heads, irreps):
    nq, nk = [rows, 20], [200, 70]
    attn = layers.CrossAttention(irreps, heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, heads, nq, nk, dtype)
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))
    # scores of some hundreds, rising along the context: every tile moves the running maximum
    k = k + (8 * torch.arange(270, device="cuda")[:, None] / 200).to(k.dtype)
    q = q + 20
    q[:3] = -q[:3]                                    # and falling for some rows
    out, lse = attn.forward(b, q, k, v, need_lse=True)
    torch.cuda.synchronize()
    ro, rl = ol.attn_forward(irreps, heads, heads, ptr_of(nq), ptr_of(nk), host(q), host(k), host(v), None, attn.scale)
    # a score of size s carries s * 2^-23 of rounding from each of its sums' steps: some 1e-4 of a weight at s = 1000
    tol = 2e-3 if dtype == "f32" else TOL[dtype]
    assert rel_err(host(out), ro) <= tol and np.abs(host(lse) - rl).max() <= 4e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_negative_and_zero_scale(dtype):
    irreps, nq, nk = "32x0e+8x1o", [40, 300, 1], [70, 33, 100]
    attn = layers.CrossAttention(irreps, 4, dtype=dtype)
    q, k, v, g = inputs(irreps, 4, 4, nq, nk, dtype)
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))
    for scale in (-0.4, 0.0, 30.0):
        out, lse = attn.forward(b, q, k, v, scale=scale, need_lse=True)
        grads = attn.backward(b, q, k, v, out, lse, g, scale=scale)
        torch.cuda.synchronize()
        args = (irreps, 4, 4, ptr_of(nq), ptr_of(nk), host(q), host(k), host(v), None, scale)
        ro, rl = ol.attn_forward(*args)
        assert rel_err(host(out), ro) <= (TOL[dtype] if scale < 1 else max(TOL[dtype], 2e-3))
        if scale > 1:
            continue                                  # (scores of hundreds: as above)
        for x, y in zip(grads, ol.attn_backward(*args, host(g))):
            assert np.abs(host(x) - y).max() <= TOL[dtype] * max(np.abs(y).max(), 0.1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_and_misaligned_rows(dtype):
    irreps, heads, nq, nk = "32x0e+16x1o", 4, [40, 50], [70, 20]
    attn = layers.CrossAttention(irreps, heads, dtype=dtype)
    q, k, v, g = inputs(irreps, heads, heads, nq, nk, dtype)
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))
    out, lse = attn.forward(b, q, k, v, need_lse=True)
    want = (out, lse) + attn.backward(b, q, k, v, out, lse, g)
    d = attn.dim_kv
    for pad in (0, 16, 3):                            # a slice of a joint row; a wider, aligned row; a misaligned one
        kv = torch.zeros((sum(nk), 2 * d + pad), dtype=torch_dtype(dtype), device="cuda")
        k2, v2 = kv[:, :d], kv[:, d + pad:]
        k2.copy_(k)
        v2.copy_(v)
        wide = torch.zeros((sum(nq), 2 * attn.dim_q + pad), dtype=torch_dtype(dtype), device="cuda")
        q2, g2 = wide[:, pad:pad + attn.dim_q], wide[:, pad + attn.dim_q:]
        q2.copy_(q)
        g2.copy_(g)
        out2, lse2 = attn.forward(b, q2, k2, v2, need_lse=True)
        got = (out2, lse2) + attn.backward(b, q2, k2, v2, out2, lse2, g2)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_gradients_match_differences():
    # the fp32 forward's own differences: step 1e-2 leaves 1e-4 of truncation and 1e-7 / 1e-2 of rounding
    irreps, heads, kv_heads, nq, nk = "8x0e+4x1o", 4, 2, [5, 2], [7, 40]
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype="f32")
    q, k, v, g = inputs(irreps, heads, kv_heads, nq, nk, "f32", seed=3)
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))
    out, lse = attn.forward(b, q, k, v, need_lse=True)
    grads = attn.backward(b, q, k, v, out, lse, g)
    f = lambda *a: (attn.forward(b, *a).double() * g.double()).sum().item()
    for i in range(3):
        args = [q, k, v]
        d = dev(np.random.default_rng(40 + i).standard_normal(args[i].shape), "f32")
        h = 1e-2
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * d, args[i] - h * d
        num = (f(*up) - f(*dn)) / (2 * h)
        assert abs(num - (grads[i] * d).sum().item()) < 5e-3 * (1 + abs(num))


def test_only_some_gradients():
    irreps, nq, nk = "128x0e+128x1o+128x2e+128x3o", [40], [50]
    for dtype in ("f32", "bf16"):
        attn = layers.CrossAttention(irreps, 8, dtype=dtype)
        q, k, v, g = inputs(irreps, 8, 8, nq, nk, dtype)
        b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))
        out, lse = attn.forward(b, q, k, v, need_lse=True)
        full = attn.backward(b, q, k, v, out, lse, g)
        for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
            part = attn.backward(b, q, k, v, out, lse, g, need=need)
            for n, x, y in zip(need, part, full):
                assert (x is None) if not n else torch.equal(x, y)


def test_packed_context_serves_other_query_counts():
    irreps, heads, kv_heads, nk = "64x0e+32x1o", 8, 2, [300, 0, 45]
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype="bf16")
    ks = layers.Samples(ptr_of(nk))
    q, k, v, _ = inputs(irreps, heads, kv_heads, [20, 7, 90], nk, "bf16")
    big = attn.batch(layers.Samples(ptr_of([20, 7, 90])), ks)
    one = attn.batch(layers.Samples(ptr_of([1, 1, 1])), ks)
    ctx = attn.pack(one, k, v)
    assert torch.equal(attn.forward_packed(big, q, ctx), attn.forward(big, q, k, v))
    step = q[[0, 20, 27]].contiguous()
    got = attn.forward_packed(one, step, ctx)
    torch.cuda.synchronize()
    ref, _ = ol.attn_forward(irreps, heads, kv_heads, [0, 1, 2, 3], ptr_of(nk), host(step), host(k), host(v), None,
                             attn.scale)
    assert rel_err(host(got), ref) <= TOL["bf16"]


def test_empty_batches():
    attn = layers.CrossAttention("16x0e", 2)
    for qp, kp in (([0], [0]), ([0, 0], [0, 5]), ([0, 3], [0, 0])):
        b = attn.batch(layers.Samples(qp), layers.Samples(kp))
        q = torch.ones((qp[-1], 16), device="cuda")
        k = torch.ones((kp[-1], 16), device="cuda")
        out, lse = attn.forward(b, q, k, k, need_lse=True)
        dq, dk, dv = attn.backward(b, q, k, k, out, lse, q)
        torch.cuda.synchronize()
        assert all(torch.all(t == 0) for t in (out, dq, dk, dv)) and torch.all(torch.isinf(lse))


def test_side_stream_and_graph():
    irreps, heads, nq, nk = "32x0e+32x1o", 4, [100, 1], [500, 3000]
    attn = layers.CrossAttention(irreps, heads, dtype="bf16")
    q, k, v, g = inputs(irreps, heads, heads, nq, nk, "bf16")
    b = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)))

    def step(q, k, v, g):
        out, lse = attn.forward(b, q, k, v, need_lse=True)
        return (out, lse) + attn.backward(b, q, k, v, out, lse, g)

    want = step(q, k, v, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(q, k, v, g)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    qs = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(qs, k, v, g)
    for i in range(3):
        qs.copy_(q * (1 + i))
        graph.replay()
        ref = step(qs, k, v, g)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(res, ref))


def test_refusals():
    attn = layers.CrossAttention("16x0e+8x1o", 4)
    other = layers.CrossAttention("16x0e+8x1o", 4)
    s3, s5 = layers.Samples([0, 3]), layers.Samples([0, 5])
    b = attn.batch(s3, s5)
    q, k = torch.zeros((3, attn.dim_q), device="cuda"), torch.zeros((5, attn.dim_kv), device="cuda")
    for bad in (lambda: attn.forward(b, q[:2], k, k), lambda: attn.forward(b, q, k.half(), k),
                lambda: attn.forward(b, q, k, k.cpu()), lambda: attn.forward(b, q, k[:, ::2], k),
                lambda: attn.forward(b, q, k, k, key_mask=torch.ones(4, dtype=torch.bool, device="cuda")),
                lambda: attn.forward(b, q, k, k, key_mask=torch.ones(5, device="cuda")),
                lambda: other.forward(b, q, k, k)):
        with pytest.raises(ValueError):
            bad()
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    for status, bad in ((1, lambda: attn.forward(b, q, k, k, scale=float("inf"))),
                        (5, lambda: attn.forward(b, q, k, k, ws=small)),
                        (5, lambda: attn.pack(b, k, k, out=small)),
                        (5, lambda: attn.forward_packed(b, q, small)),
                        (1, lambda: attn.batch(s3, layers.Samples([0, 2, 5])))):
        with pytest.raises(cgtp.CgtpError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("irreps,heads,kv_heads,nq", [
    ("35x0e+21x1o+7x2e", 7, 1, [1, 70, 5]),                         # few rows; ordinary
    ("128x0e+128x1o", 4, 2, [3, 300, 40]),                          # 64-row waves
    ("128x0e+128x1o+128x2e", 8, 4, [50, 140, 1]),
])
def test_rows_that_see_one_key(irreps, heads, kv_heads, nq):
    """bf16: such a row is its value exactly, and its score gradients cancel.

    out = (w v) / w with the same rounded weight w, v to fp32's last bits, rounded to v.
    grad_q = scale P (dP - delta) k, dP and delta the same D products g v summed in
    fp32 in two orders, each sum off by at most D 2^-24 sum |g v| from the exact one.
    grad_k adds such terms over queries and heads. P is 1 to 2e-5, and rounding to
    bf16 (twice) adds 2^-8 of the result: a factor of 1.1 covers both."""
    nk, rng = [40, 65, 3], np.random.default_rng(23)
    q, k, v, g = inputs(irreps, heads, kv_heads, nq, nk, "bf16", seed=21)
    qp, kp = ptr_of(nq), ptr_of(nk)
    seen = [rng.integers(a, b) for a, b in zip(kp[:-1], kp[1:])]
    mask = torch.zeros(kp[-1], dtype=torch.bool)
    mask[seen] = True
    attn = layers.CrossAttention(irreps, heads, kv_heads, dtype="bf16")
    batch = attn.batch(layers.Samples(qp), layers.Samples(kp))
    out, lse = attn.forward(batch, q, k, v, key_mask=mask.cuda(), need_lse=True)
    dq, dk, _ = (host(t) for t in attn.backward(batch, q, k, v, out, lse, g, key_mask=mask.cuda()))
    hq, hk, hv, hg, ho = host(q), host(k), host(v), host(g), host(out)
    kvi = ol.kv_irreps(irreps, heads, kv_heads)
    for s, j in enumerate(seen):
        for h in range(heads):
            rows = np.ix_(np.arange(qp[s], qp[s + 1]), ol.head_columns(irreps, heads, h))
            cols = ol.head_columns(kvi, kv_heads, h * kv_heads // heads)
            assert np.array_equal(ho[rows], np.broadcast_to(hv[j, cols], ho[rows].shape))
            sums = 2 * len(cols) * 2.0 ** -24 * np.abs(hg[rows] * hv[j, cols]).sum(1, keepdims=True)
            assert (np.abs(dq[rows]) <= 1.1 * attn.scale * sums * np.abs(hk[j, cols])).all()
        for h in range(kv_heads):
            cols, bound = ol.head_columns(kvi, kv_heads, h), 0.0
            for hh in range(h * heads // kv_heads, (h + 1) * heads // kv_heads):
                rows = np.ix_(np.arange(qp[s], qp[s + 1]), ol.head_columns(irreps, heads, hh))
                sums = 2 * len(cols) * 2.0 ** -24 * np.abs(hg[rows] * hv[j, cols]).sum(1, keepdims=True)
                bound = bound + (sums * np.abs(hq[rows])).sum(0)
            assert (np.abs(dk[j, cols]) <= 1.1 * attn.scale * bound).all()
