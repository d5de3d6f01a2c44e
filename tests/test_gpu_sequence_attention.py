"""GPU attention along sequences against the fp64 oracle: causal batches (whole
prompts, next rows after earlier ones, contexts shorter than the queries), rows that
all samples share, both together; ragged and empty samples, one token to long ones,
grouped heads, odd channel counts, head sizes up to 256, masks that leave rows
empty, infinities and NaN where a query does not see them, strided rows, splits, the
packed form; gradients also against differences; streams, graph capture, refusals."""

import numpy as np
import pytest

from oracle import layers as ol
from tests.gpu_util import TOL, dev, host, rel_err, torch_dtype
from tests.test_gpu_attention import inputs, ptr_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

# (irreps, heads, kv heads, query lengths, own context lengths, causal, shared rows)
CASES = [
    ("8x0e", 1, 1, [1], [1], True, 0),
    ("32x0e+32x1o+32x2e", 4, 4, [9, 21, 0, 1], [9, 21, 0, 1], True, 0),
    ("10x0e+6x1o", 2, 1, [3, 70, 31, 32, 33], [3, 70, 31, 32, 33], True, 0),     # element-wise rows
    ("35x0e+21x1o+7x2e", 7, 1, [40, 1, 13], [40, 1, 13], True, 0),               # 7 heads share a context head
    ("64x0e", 2, 2, [129, 32, 64], [129, 32, 64], True, 0),
    ("64x0e", 8, 2, [20, 5], [120, 37], True, 0),                                # next rows after earlier ones
    ("64x0e", 2, 2, [70, 10, 5, 40], [33, 2, 0, 39], True, 0),                   # queries that see no own key
    ("128x0e+128x1o", 4, 4, [300], [300], True, 0),
    ("128x0e+128x1o", 16, 4, [180, 3], [181, 40], True, 0),                      # head of 32
    ("128x0e+128x1o+128x2e", 8, 4, [50, 140], [50, 140], True, 0),               # 144, padded to 160
    ("24x0e+24x1o+24x2e+24x3o", 2, 1, [33], [50], True, 0),                      # 192
    ("14x0e+14x1o+14x2e+14x3o", 1, 1, [70], [70], True, 0),                      # 224
    ("128x0e+128x1o+128x2e+128x3o", 8, 8, [70], [70], True, 0),                  # 256
    ("128x0e+128x1o+128x2e+128x3o", 16, 4, [1, 1, 1], [700, 1, 1500], True, 0),  # single tokens, split
    ("16x0e", 4, 2, [700, 90], [700, 1500], True, 0),                            # all kernels, splits
    ("64x0e", 1, 1, [600, 1], [600, 1], True, 0),                                # 64 rows a wave
    ("8x0e", 1, 1, [1], [0], False, 1),
    ("32x0e+32x1o+32x2e", 4, 2, [3, 1, 0, 8], [0, 20, 5, 7], False, 50),         # few rows: joined by rows
    ("32x0e+32x1o+32x2e", 4, 2, [3, 1, 0, 8], [3, 20, 5, 7], True, 50),
    ("64x0e", 8, 1, [1] * 40, [1] * 20 + [40] * 20, True, 333),                  # single tokens
    ("35x0e+21x1o+7x2e", 7, 1, [40, 1, 9], [31, 0, 12], False, 33),
    ("128x0e+128x1o", 4, 4, [130, 20], [10, 64], False, 300),
    ("128x0e+128x1o+128x2e", 8, 4, [50, 70], [50, 70], True, 64),
    ("128x0e+128x1o+128x2e+128x3o", 16, 4, [1, 2, 1], [70, 2, 40], True, 500),
    ("16x0e", 4, 2, [300, 1, 9], [300, 1, 40], True, 1000),
    ("64x0e", 1, 1, [300, 270, 1], [300, 0, 70], True, 200),                     # 64 rows a wave
    ("64x0e", 2, 2, [70, 10, 5], [33, 2, 0], True, 3),
    ("64x0e", 1, 1, [1, 300, 40, 0, 31], [1, 300, 40, 0, 31], True, 0),          # one kernel for all
    ("64x0e", 1, 1, [1, 300, 40], [1, 300, 900], True, 0),                       # two
]


def check(attn, case, dtype, q, k, v, g, mask=None, refs=None):
    irreps, heads, kv_heads, nq, nk, causal, shared = case
    qp, kp = ptr_of(nq), ptr_of(nk)
    batch = attn.batch(layers.Samples(qp), layers.Samples(kp), causal=causal, shared=shared)
    assert batch.nk == shared + sum(nk)
    out, lse = attn.forward(batch, q, k, v, key_mask=mask, need_lse=True)
    torch.cuda.synchronize()
    grads = attn.backward(batch, q, k, v, out, lse, g, key_mask=mask)
    torch.cuda.synchronize()
    packed = attn.forward_packed(batch, q, attn.pack(batch, k, v, key_mask=mask))
    torch.cuda.synchronize()
    hm = None if mask is None else mask.cpu().numpy()
    hq, hk, hv, hg = refs or (host(q), host(k), host(v), host(g))
    args = (irreps, heads, kv_heads, qp, kp, hq, hk, hv, hm, attn.scale)
    ro, rl = ol.seq_forward(*args, causal, shared)
    rg = ol.seq_backward(*args, hg, causal, shared)
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


def make(case, dtype, seed=0):
    irreps, heads, kv_heads, nq, nk, causal, shared = case
    return (layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype),) + tuple(
        inputs(irreps, heads, kv_heads, nq, [shared] + list(nk), dtype, seed))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_sequence_attention(case, dtype):
    print("sequence attention", case, dtype, flush=True)
    attn, q, k, v, g = make(case, dtype)
    a = check(attn, case, dtype, q, k, v, g)
    b = check(attn, case, dtype, q, k, v, g)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,heads,kv_heads,nq,nk,causal,shared", [
    ("128x0e+128x1o", 8, 2, [1, 2, 1, 0] * 16, [1, 20, 0, 7] * 16, True, 9000),
    ("128x0e+128x1o+128x2e+128x3o", 16, 4, [1] * 40, [3] * 40, False, 8100),
    ("128x0e+128x1o+128x2e+128x3o", 16, 16, [1] * 30, [1, 300, 40] * 10, True, 4000)])
def test_few_rows_of_many_samples_on_long_shared_rows(irreps, heads, kv_heads, nq, nk, causal, shared, dtype):
    """(these go against the shared rows together) against the definition in 64 bits"""
    attn, q, k, v, g = make((irreps, heads, kv_heads, nq, nk, causal, shared), dtype)
    qp, kp = ptr_of(nq), ptr_of(nk)
    mask = torch.rand(shared + sum(nk), device="cuda", generator=torch.Generator("cuda").manual_seed(3)) < 0.9
    batch = attn.batch(layers.Samples(qp), layers.Samples(kp), causal=causal, shared=shared)
    out, lse = attn.forward(batch, q, k, v, key_mask=mask, need_lse=True)
    again = attn.forward(batch, q, k, v, key_mask=mask)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    want, want_lse = torch.zeros(out.shape, dtype=torch.float64, device="cuda"), torch.zeros_like(lse, dtype=torch.float64)
    kvi = ol.kv_irreps(irreps, heads, kv_heads)
    for h in range(heads):
        qc = torch.from_numpy(ol.head_columns(irreps, heads, h)).cuda()
        kc = torch.from_numpy(ol.head_columns(kvi, kv_heads, h * kv_heads // heads)).cuda()
        qh, kh, vh = q[:, qc].double(), k[:, kc].double(), v[:, kc].double()
        for s in range(len(nq)):
            for i in range(nq[s]):
                n = max(0, i + nk[s] - nq[s] + 1) if causal else nk[s]
                keys = torch.cat([torch.arange(shared, device="cuda"), shared + kp[s] + torch.arange(n, device="cuda")])
                keys = keys[mask[keys]]
                w = kh[keys] @ qh[qp[s] + i] * attn.scale
                want[qp[s] + i, qc] = torch.softmax(w, 0) @ vh[keys]
                want_lse[qp[s] + i, h] = torch.logsumexp(w, 0)
    assert rel_err(host(out), want.cpu().numpy()) <= TOL[dtype]
    assert (lse.double() - want_lse).abs().max().item() <= 2e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nq,nk,causal,shared", [([40, 3, 70], [90, 33, 64], True, 0), ([40, 3, 70], [90, 33, 64], True, 40),
                                                 ([3, 1, 2], [90, 33, 64], True, 40), ([3, 1, 2], [90, 33, 64], False, 40)])
def test_masks_with_nan_and_inf_in_masked_places(dtype, nq, nk, causal, shared):
    case = ("32x0e+16x1o", 4, 2, nq, nk, causal, shared)
    attn, q, k, v, g = make(case, dtype)
    mask = torch.from_numpy(np.random.default_rng(5).random(shared + sum(nk)) < 0.6).cuda()
    mask[:shared] = False                             # only own keys count, and the second sample has none left
    mask[shared + 90:shared + 123] = False
    mask[-1], mask[shared] = True, False
    refs = [host(t) for t in (q, k, v, g)]
    for t, bad in ((k, float("nan")), (v, float("inf"))):
        t[~mask] = bad
    refs[1][~mask.cpu().numpy()] = 0
    refs[2][~mask.cpu().numpy()] = 0
    lo, hi = nq[0], nq[0] + nq[1]
    g[lo:hi] = float("nan")                           # gradients of rows that saw nothing do not spread
    refs[3][lo:hi] = 0
    for m in (mask, mask.to(torch.uint8) * 3):
        out, lse, dq, dk, dv = check(attn, case, dtype, q, k, v, g, mask=m, refs=refs)
        assert torch.all(out[lo:hi] == 0) and torch.all(dq[lo:hi] == 0) and torch.all(torch.isinf(lse[lo:hi]))
        assert torch.all(dk[~mask] == 0) and torch.all(dv[~mask] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,heads,kv_heads,lens,shared", [
    ("32x0e+16x1o", 4, 2, [70, 9], 0), ("32x0e+16x1o", 4, 2, [5, 9], 40), ("64x0e", 1, 1, [500, 3], 33),
    ("64x0e", 2, 2, [1500], 0), ("10x0e+6x1o", 2, 1, [40, 9], 0)])
def test_what_later_keys_hold_does_not_reach_earlier_queries(irreps, heads, kv_heads, lens, shared, dtype):
    """NaN and infinities in a token's key or value: the tokens before it keep their out
    and lse, and behind it follows what the formula gives."""
    case = (irreps, heads, kv_heads, lens, lens, True, shared)
    attn, q, k, v, g = make(case, dtype)
    samples = layers.Samples(ptr_of(lens))
    batch = attn.batch(samples, samples, causal=True, shared=shared)
    want, want_lse = attn.forward(batch, q, k, v, need_lse=True)
    at = lens[0] - 4
    for tensor, bad in ((v, float("inf")), (v, float("nan")), (k, float("nan"))):
        x, y = k.clone(), v.clone()
        (x if tensor is k else y)[shared + at, 3] = bad
        out, lse = attn.forward(batch, q, x, y, need_lse=True)
        torch.cuda.synchronize()
        rest = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
        rest[at:lens[0]] = False
        # Not bit by bit: a row formed again adds its keys in another order, and a NaN among the keys' norms makes
        # the kernel keep a running maximum, another reference. Scores of up to 20 (log2) less a reference of up to
        # 40 round by 60 * 2^-24 at most, twice, so weights and their sums move by 2 * 60 * 2^-24 * ln 2 = 5e-6
        # relative; in bf16 a weight may then fall to the neighbouring number (2^-8), and so may the result.
        big, top = y[torch.isfinite(y)].float().abs().max().item(), want.float().abs().max().item()
        tol = 1e-5 * big if dtype == "f32" else 2.0 ** -8 * (big + top)
        assert (out[rest].float() - want[rest].float()).abs().max().item() <= tol
        assert (lse[rest] - want_lse[rest]).abs().max().item() <= 1e-5
        behind = host(out[at:lens[0]])
        if tensor is v:                               # of the heads that read that column alone
            cols = [c for h in range(heads) for c, d in zip(ol.head_columns(irreps, heads, h), ol.head_columns(
                ol.kv_irreps(irreps, heads, kv_heads), kv_heads, h * kv_heads // heads)) if d == 3]
            clean = np.setdiff1d(np.arange(attn.dim_q), cols)
            assert not np.isfinite(behind[:, cols]).any() and np.isfinite(behind[:, clean]).all()
            assert not np.isinf(bad) or np.all(behind[:, cols] == np.inf)
            assert torch.equal(lse, want_lse)     # the values have no part in it
        else:
            assert np.isnan(behind).any(1).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,heads,kv_heads,lens,shared", [
    ("32x0e+16x1o", 4, 2, [70, 9], 0), ("64x0e", 1, 1, [500, 3], 33), ("64x0e", 2, 2, [1500], 0),
    ("128x0e+128x1o+128x2e", 8, 4, [50, 90], 0), ("10x0e+6x1o", 2, 1, [40, 9], 7)])
def test_nan_does_not_reach_gradients_that_do_not_depend_on_it(irreps, heads, kv_heads, lens, shared, dtype):
    case = (irreps, heads, kv_heads, lens, lens, True, shared)
    clean = make(case, dtype)
    attn = clean[0]
    samples = layers.Samples(ptr_of(lens))
    batch = attn.batch(samples, samples, causal=True, shared=shared)
    at = lens[0] - 10                                 # tokens before and behind it share its tile

    def grads(q, k, v, g):
        out, lse = attn.forward(batch, q, k, v, need_lse=True)
        return attn.backward(batch, q, k, v, out, lse, g)

    want = grads(*clean[1:])
    n = sum(lens)
    rows, keys = torch.arange(n, device="cuda"), torch.arange(shared + n, device="cuda") - shared
    for which in range(4):                            # q, k, v, grad_out of token `at`
        args = [t.clone() for t in clean[1:]]
        args[which][at + (shared if which in (1, 2) else 0), 3] = float("nan")
        got = grads(*args)
        torch.cuda.synchronize()
        if which in (0, 3):                           # a query reaches its own gradient, and the keys that it sees
            free = (rows != at, keys > at, keys > at)
        else:                                         # a key reaches the queries that see it, and by them all their keys
            free = (rows < at, keys >= lens[0], keys >= lens[0])
            free = ((rows < at) | (rows >= lens[0]),) + free[1:]
        for i, (a, b, m) in enumerate(zip(got, want, free)):
            if m.any():
                # as two results of one type, each off by its tolerance against the formula
                scale = b.float().abs().max().item()
                assert (a[m].float() - b[m].float()).abs().max().item() <= 2 * TOL[dtype] * scale, (which, i)
        bad = (got[0][at], got[0][at:lens[0]], got[0][at:lens[0]], got[1][shared])[which]
        assert torch.isnan(bad).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shared", [0, 37])
def test_strided_and_misaligned_rows(dtype, shared):
    case = ("32x0e+16x1o", 4, 4, [40, 50], [40, 50], True, shared)
    attn, q, k, v, g = make(case, dtype)
    s = layers.Samples([0, 40, 90])
    b = attn.batch(s, s, causal=True, shared=shared)
    out, lse = attn.forward(b, q, k, v, need_lse=True)
    want = (out, lse) + attn.backward(b, q, k, v, out, lse, g)
    d, n = attn.dim_kv, shared + 90
    for pad in (0, 16, 3):                            # a slice of a joint row; a wider, aligned row; a misaligned one
        kv = torch.zeros((n, 2 * d + pad), dtype=torch_dtype(dtype), device="cuda")
        k2, v2 = kv[:, :d], kv[:, d + pad:]
        k2.copy_(k)
        v2.copy_(v)
        wide = torch.zeros((90, 2 * attn.dim_q + pad), dtype=torch_dtype(dtype), device="cuda")
        q2, g2 = wide[:, pad:pad + attn.dim_q], wide[:, pad + attn.dim_q:]
        q2.copy_(q)
        g2.copy_(g)
        out2, lse2 = attn.forward(b, q2, k2, v2, need_lse=True)
        got = (out2, lse2) + attn.backward(b, q2, k2, v2, out2, lse2, g2)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("causal,shared", [(True, 0), (True, 5), (False, 5)])
def test_gradients_match_differences(causal, shared):
    # the fp32 forward's own differences: step 1e-2 leaves 1e-4 of truncation and 1e-7 / 1e-2 of rounding
    case = ("8x0e+4x1o", 4, 2, [5, 2, 4], [7, 40, 4], causal, shared)
    attn, q, k, v, g = make(case, "f32", seed=3)
    b = attn.batch(layers.Samples(ptr_of(case[3])), layers.Samples(ptr_of(case[4])), causal=causal, shared=shared)
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
    case = ("128x0e+128x1o", 4, 2, [40, 9], [40, 9], True, 20)
    for dtype in ("f32", "bf16"):
        attn, q, k, v, g = make(case, dtype)
        s = layers.Samples([0, 40, 49])
        b = attn.batch(s, s, causal=True, shared=20)
        out, lse = attn.forward(b, q, k, v, need_lse=True)
        full = attn.backward(b, q, k, v, out, lse, g)
        for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
            some = attn.backward(b, q, k, v, out, lse, g, need=need)
            assert all((x is None) if not n else torch.equal(x, y) for n, x, y in zip(need, some, full))


def test_large_scores_and_signs_of_the_scale():
    case = ("64x0e", 2, 2, [300, 20], [300, 20], True, 40)
    for dtype in ("f32", "bf16"):
        attn, q, k, v, g = make(case, dtype)
        s = layers.Samples([0, 300, 320])
        b = attn.batch(s, s, causal=True, shared=40)
        k2 = k + (8 * torch.arange(360, device="cuda")[:, None] / 200).to(k.dtype)
        for scale, keys in ((None, k2), (-0.4, k), (0.0, k)):
            x = q + 20 if keys is k2 else q
            out, lse = attn.forward(b, x, keys, v, scale=scale, need_lse=True)
            torch.cuda.synchronize()
            ro, rl = ol.seq_forward("64x0e", 2, 2, [0, 300, 320], [0, 300, 320], host(x), host(keys), host(v), None,
                                    attn.scale if scale is None else scale, True, 40)
            # a score of size s carries s * 2^-23 of rounding from each of its sums' steps: some 1e-4 of a weight at s = 1000
            tol = 2e-3 if dtype == "f32" and keys is k2 else TOL[dtype]
            assert rel_err(host(out), ro) <= tol
            assert np.abs(host(lse) - rl).max() <= (4e-3 if keys is k2 else 2e-5)


def test_the_whole_and_the_causal_batch_agree_where_they_mean_the_same():
    """One query a sample sees all of its context in a causal batch; shared rows are as if
    each sample had them at the start of its own."""
    for dtype in ("f32", "bf16"):
        nk = [70, 3, 500]
        attn, q, k, v, g = make(("64x0e", 4, 2, [1, 1, 1], nk, True, 0), dtype)
        one, ctx = layers.Samples([0, 1, 2, 3]), layers.Samples(ptr_of(nk))
        a = attn.forward(attn.batch(one, ctx), q, k, v)
        b = attn.forward(attn.batch(one, ctx, causal=True), q, k, v)
        assert torch.equal(a, b)
        shared = 64
        nq = [40, 80]
        attn, q, k, v, g = make(("64x0e", 4, 2, nq, [30, 50], False, shared), dtype)
        c = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples([0, 30, 80]), shared=shared)
        twice = lambda t: torch.cat([t[:shared], t[shared:shared + 30], t[:shared], t[shared + 30:]])
        d = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples([0, shared + 30, 2 * shared + 80]))
        x, xl = attn.forward(c, q, k, v, need_lse=True)
        y, yl = attn.forward(d, q, twice(k), twice(v), need_lse=True)
        # the same sums in another split at most
        assert rel_err(host(x), host(y)) <= TOL[dtype] and (xl - yl).abs().max().item() <= 2e-5
        gx = attn.backward(c, q, k, v, x, xl, g)
        gy = attn.backward(d, q, twice(k), twice(v), y, yl, g)
        assert rel_err(host(gx[0]), host(gy[0])) <= TOL[dtype]
        for p, r in zip(gx[1:], gy[1:]):
            r = r.double()
            first, second = r[:shared + 30], r[shared + 30:]
            sums = torch.cat([first[:shared] + second[:shared], first[shared:], second[shared:]])
            assert rel_err(host(p), host(sums)) <= TOL[dtype]


@pytest.mark.parametrize("shared", [0, 40])
def test_captured_training_step_and_streams(shared):
    case = ("32x0e+16x1o", 4, 2, [300, 5, 40], [300, 5, 40], True, shared)
    attn, q, k, v, g = make(case, "bf16")
    s = layers.Samples(ptr_of(case[3]))
    b = attn.batch(s, s, causal=True, shared=shared)

    def step():
        out, lse = attn.forward(b, q, k, v, need_lse=True)
        return (out, lse) + attn.backward(b, q, k, v, out, lse, g)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2, 3):
        fresh = inputs(case[0], 4, 2, case[3], [shared] + case[4], "bf16", seed)
        for t, f in zip((q, k, v, g), fresh):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_a_packed_context_serves_other_queries():
    case = ("64x0e", 4, 2, [9, 40], [90, 70], True, 33)
    for dtype in ("f32", "bf16"):
        attn, q, k, v, g = make(case, dtype)
        ctx = layers.Samples([0, 90, 160])
        a = attn.batch(layers.Samples([0, 9, 49]), ctx, causal=True, shared=33)
        b = attn.batch(layers.Samples([0, 1, 2]), ctx, causal=True, shared=33)
        packed = attn.pack(a, k, v)
        whole = attn.forward_packed(a, q, packed)
        last = attn.forward_packed(b, q[[8, 48]].contiguous(), packed)
        torch.cuda.synchronize()
        # (the same keys by another kernel: its sums' order)
        assert rel_err(host(last), host(whole[[8, 48]])) <= TOL[dtype]


def test_batches_without_samples_or_rows():
    attn = layers.CrossAttention("32x0e", 4)
    none, empty = layers.Samples([0]), layers.Samples([0, 0, 0])
    k = torch.ones((3, 32), device="cuda")
    for samples in (none, empty):
        for causal in (False, True):
            b = attn.batch(samples, samples, causal=causal, shared=3)
            q = torch.zeros((0, 32), device="cuda")
            out, lse = attn.forward(b, q, k, k, need_lse=True)
            dq, dk, dv = attn.backward(b, q, k, k, out, lse, q)
            torch.cuda.synchronize()
            assert out.shape == (0, 32) and dq.shape == (0, 32)
            assert torch.all(dk == 0) and torch.all(dv == 0)      # nobody reads the shared rows


def test_refusals():
    attn = layers.CrossAttention("32x0e", 4)
    s, t = layers.Samples([0, 5]), layers.Samples([0, 3, 7])
    with pytest.raises(cgtp.CgtpError) as e:
        attn.batch(s, t, causal=True)
    assert e.value.status == 1
    with pytest.raises(cgtp.CgtpError) as e:
        attn.batch(s, s, shared=-1)
    assert e.value.status == 1
    with pytest.raises(cgtp.CgtpError) as e:
        attn.batch(s, s, shared=1 << 40)
    assert e.value.status == 3
    with pytest.raises(cgtp.CgtpError) as e:
        attn.batch(s, s, shared=(1 << 31) - 3)
    assert e.value.status == 3
    b = attn.batch(s, s, causal=True, shared=4)
    q, k = torch.zeros((5, 32), device="cuda"), torch.zeros((9, 32), device="cuda")
    attn.forward(b, q, k, k)
    for bad in (q, torch.zeros((10, 32), device="cuda"), k.bfloat16()):
        with pytest.raises(ValueError):
            attn.forward(b, q, bad, k)
    with pytest.raises(ValueError):
        attn.forward(b, q, k, k, key_mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(cgtp.CgtpError) as e:
        attn.forward(b, q, k, k, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status not in (0, 1, 3)
