"""GPU attention along sequences where sums and references are at their ends: rows of
which some parts see no key, with scores far below zero."""

import numpy as np
import pytest

from oracle import layers as ol
from tests.gpu_util import TOL, dev, host, rel_err
from tests.test_gpu_attention import ptr_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

# A score is a sum of 32 products of size 6: rounding leaves at most 32 * 2^-24 * 196 = 3.7e-4 of
# it, twice that of a weight and of its share in the result, so 2e-3 of the largest value covers
# fp32; bf16 adds its own rounding. An lse is off by as much as its scores, 1e-3 at most.
FAR_TOL = {"f32": 2e-3, "bf16": TOL["bf16"]}
FAR_LSE = 1e-3


def far_rows(rng, nq, nk, d, dtype):
    """Queries and keys whose products are near -196, and values."""
    base = 14.0 / np.sqrt(32)
    heads = d // 32
    q = dev(-base + 0.1 * rng.standard_normal((nq, d)), dtype)
    k, v = dev(base + 0.1 * rng.standard_normal((nk, d)), dtype), dev(rng.standard_normal((nk, d)), dtype)
    return heads, q, k, v


# Where the shared rows are seen (of 4500): parts without a key in front, behind and on both sides.
SEEN = [(0, 100), (150, 250), (400, 500), (2200, 2300), (3000, 3100), (4400, 4500)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal,scale", [(False, 1.0), (True, 1.0), (True, -1.0)])
@pytest.mark.parametrize("seen", SEEN)
def test_few_rows_whose_parts_see_no_shared_key(seen, causal, scale, dtype):
    """Samples of a tile at most on long shared rows, joined by rows: 1 - 16 rows a sample,
    with no own keys, masked ones, and some that count."""
    shared, nq = 4500, [1] * 150 + [2] * 30 + [9] * 10 + [16] * 10
    nk = [(0, 3, 0, 40)[s % 4] for s in range(len(nq))]
    rng = np.random.default_rng(41)
    heads, q, k, v = far_rows(rng, sum(nq), shared + sum(nk), 128, dtype)
    attn = layers.CrossAttention("128x0e", heads, dtype=dtype)
    qp, kp = ptr_of(nq), ptr_of(nk)
    mask = torch.zeros(shared + sum(nk), dtype=torch.bool, device="cuda")
    mask[seen[0]:seen[1]] = True
    for s in range(3, len(nk), 8):                            # own keys of every other sample that has 40
        mask[shared + kp[s]:shared + kp[s + 1]] = True
    batch = attn.batch(layers.Samples(qp), layers.Samples(kp), causal=causal, shared=shared)
    out, lse = attn.forward(batch, q, k, v, scale=scale, key_mask=mask, need_lse=True)
    torch.cuda.synchronize()
    hm = mask.cpu().numpy()
    ro, rl = ol.seq_forward("128x0e", heads, heads, qp, kp, host(q), host(k), host(v), hm, scale, causal, shared)
    assert np.isfinite(host(out)).all() and np.isfinite(host(lse)).all()
    assert np.abs(rl).min() > 150.0
    assert rel_err(host(out), ro) <= FAR_TOL[dtype]
    assert np.abs(host(lse) - rl).max() <= FAR_LSE


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("seen", SEEN[:1] + SEEN[3:] + [(0, 0)])
def test_steps_behind_masked_shared_rows_with_far_scores(seen, scale, dtype):
    shared, cap = 4500, 90
    lens = [0, 5, 31, 32, 70, -1, 90, 1] * 8
    rng = np.random.default_rng(42)
    S = len(lens)
    heads, q, k, v = far_rows(rng, S, S, 128, dtype)
    attn = layers.CrossAttention("128x0e", heads, dtype=dtype)
    cache = attn.cache(S, cap, shared=shared)
    _, _, ks, vs = far_rows(rng, 1, shared + S * cap, 128, dtype)
    cache.k.copy_(ks[shared:].view(S, cap, 128))
    cache.v.copy_(vs[shared:].view(S, cap, 128))
    mask = torch.zeros(shared, dtype=torch.bool, device="cuda")
    mask[seen[0]:seen[1]] = True
    cache.share(ks[:shared], vs[:shared], key_mask=mask)
    want = ol.cache_step("128x0e", heads, heads, host(q), host(k), host(v), host(cache.k), host(cache.v), lens, scale,
                         (host(ks[:shared]), host(vs[:shared]), mask.cpu().numpy()))
    out, lse = attn.step(cache, q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale, need_lse=True)
    torch.cuda.synchronize()
    assert np.array_equal(np.isinf(host(lse)), np.isinf(want[1]))
    assert rel_err(host(out), want[0]) <= FAR_TOL[dtype]
    fin = np.isfinite(want[1])
    assert np.abs(host(lse)[fin] - want[1][fin]).max() <= FAR_LSE
    assert np.abs(want[1][fin]).min() > 150.0


# (irreps, heads, kv heads, query lengths, own context lengths, shared rows): every kernel and both ways of writing
SPECIAL = [
    ("64x0e", 2, 2, [9, 30, 1], [9, 30, 1], 0),                # one tile a sample
    ("10x0e+6x1o", 2, 1, [70, 9], [70, 9], 0),                 # element-wise rows
    ("32x0e+16x1o", 4, 2, [90, 40], [130, 40], 33),
    ("128x0e+128x1o", 4, 2, [100], [700], 0),                  # split
    ("64x0e", 1, 1, [300, 3], [300, 3], 40),                   # 64 rows a wave in bf16
    ("64x0e", 4, 1, [1, 1, 7], [400, 900, 7], 0),              # few rows, split
    ("24x0e+24x1o+24x2e+24x3o", 2, 1, [33], [50], 0),          # heads of 192
    ("128x0e+128x1o+128x2e+128x3o", 8, 4, [70], [70], 0),      # heads of 256
]


def special_inputs(case, dtype, which, seed):
    """Inputs with infinities of both signs and NaN at some elements of the tensors `which`."""
    irreps, heads, kv_heads, nq, nk, shared = case
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    rng = np.random.default_rng(seed)
    rows = (sum(nq), shared + sum(nk), shared + sum(nk), sum(nq))
    made = []
    for i, (n, d) in enumerate(zip(rows, (attn.dim_q, attn.dim_kv, attn.dim_kv, attn.dim_q))):
        x = rng.standard_normal((n, d))
        if i in which:
            count = max(1, n * d // 2000)
            # (the later a row, the more rows it is hidden from: most of them lie in the last third)
            at = np.minimum(n - 1, (n * rng.random(count) ** 0.3).astype(int))
            x[at, rng.integers(0, d, count)] = rng.choice([np.inf, -np.inf, np.nan], count)
        made.append(dev(x, dtype))
    return (attn,) + tuple(made)


def visible_pairs(case, attn):
    irreps, heads, kv_heads, nq, nk, shared = case
    kvi = ol.kv_irreps(irreps, heads, kv_heads)
    qp, kp = ptr_of(nq), ptr_of(nk)
    for s in range(len(nq)):
        keys = np.concatenate([np.arange(shared), shared + np.arange(kp[s], kp[s + 1])])
        seen = np.arange(len(keys))[None] < shared + (np.arange(nq[s]) + nk[s] - nq[s] + 1)[:, None]
        for h in range(heads):
            yield (np.arange(qp[s], qp[s + 1]), keys, seen, h, ol.head_columns(irreps, heads, h),
                   ol.head_columns(kvi, kv_heads, h * kv_heads // heads))


def sum_seen(w, x, seen):
    """sum_j w[i, j] x[j] over the pairs that are seen: what is finite and what is not, apart."""
    finite = np.isfinite(x)
    tame = np.where(finite, x, 0.0)
    out = np.where(seen, w, 0.0) @ tame
    for d in np.flatnonzero(~finite.all(0)):
        bad = ~finite[:, d]
        with np.errstate(invalid="ignore"):
            terms = np.where(seen[:, bad], w[:, bad] * x[bad, d], 0.0)
            out[:, d] += terms.sum(1)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SPECIAL)
def test_values_with_infinities_and_nan_reach_the_rows_that_see_them_alone(case, dtype):
    attn, q, k, v, _ = special_inputs(case, dtype, (2,), 51)
    irreps, heads, kv_heads, nq, nk, shared = case
    batch = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)), causal=True, shared=shared)
    out, lse = attn.forward(batch, q, k, v, need_lse=True)
    bare = attn.forward(batch, q, k, v)
    torch.cuda.synchronize()
    hq, hk, hv, got = host(q), host(k), host(v), host(out)
    want = np.zeros_like(got)
    for rows, keys, seen, h, qc, kc in visible_pairs(case, attn):
        s = np.where(seen, attn.scale * hq[np.ix_(rows, qc)] @ hk[np.ix_(keys, kc)].T, -np.inf)
        top = s.max(1, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        total = e.sum(1, keepdims=True)
        want[np.ix_(rows, qc)] = sum_seen(e / np.where(total > 0, total, 1.0), hv[np.ix_(keys, kc)], seen)
    fin = np.isfinite(want)
    assert fin.any() and not fin.all()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    assert np.abs(got[fin] - want[fin]).max() <= TOL[dtype] * np.abs(want[fin]).max()
    assert np.isfinite(host(lse)).all()
    assert torch.equal(torch.nan_to_num(bare), torch.nan_to_num(out))
    assert torch.equal(bare.isnan(), out.isnan())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", [0, 1, 2, 3])
@pytest.mark.parametrize("case", SPECIAL)
def test_gradients_beside_infinities_and_nan(case, which, dtype):
    """Of one tensor at a time (q, k, v, grad_out), from the formula over the pairs that are seen: what is
    finite there is finite and near it, and what is NaN or infinite there is not finite."""
    args = special_inputs(case, dtype, (which,), 52 + which)
    attn, q, k, v, g = args
    irreps, heads, kv_heads, nq, nk, shared = case
    batch = attn.batch(layers.Samples(ptr_of(nq)), layers.Samples(ptr_of(nk)), causal=True, shared=shared)
    out, lse = attn.forward(batch, q, k, v, need_lse=True)
    grads = [host(t) for t in attn.backward(batch, q, k, v, out, lse, g)]
    torch.cuda.synchronize()
    hq, hk, hv, hg = host(q), host(k), host(v), host(g)
    want = [np.zeros_like(t) for t in grads]
    with np.errstate(invalid="ignore", over="ignore"):
        for rows, keys, seen, h, qc, kc in visible_pairs(case, attn):
            qi, ki = np.ix_(rows, qc), np.ix_(keys, kc)
            some = seen.any(1)
            s = np.where(seen, attn.scale * hq[qi] @ hk[ki].T, -np.inf)
            top = np.where(some[:, None], s.max(1, keepdims=True), 0.0)
            e = np.where(seen, np.exp(s - top), 0.0)
            p = e / np.where(some[:, None], e.sum(1, keepdims=True), 1.0)
            o = sum_seen(p, hv[ki], seen)
            ds = np.where(seen, p * (hg[qi] @ hv[ki].T - (hg[qi] * o).sum(1, keepdims=True)) * attn.scale, 0.0)
            gi = np.where(some[:, None], hg[qi], 0.0)           # rows that see nothing have no part
            qz = np.where(some[:, None], hq[qi], 0.0)
            want[0][qi] += sum_seen(ds, hk[ki], seen)
            want[1][ki] += sum_seen(ds.T, qz, seen.T)
            want[2][ki] += sum_seen(p.T, gi, seen.T)
    for name, a, b in zip(("grad_q", "grad_k", "grad_v"), grads, want):
        fin = np.isfinite(b)
        assert not np.isfinite(a[~fin]).any(), name
        if fin.any():
            assert np.isfinite(a[fin]).all(), name
            scale = max([np.abs(b[fin]).max()] + [0.1 * np.abs(w[np.isfinite(w)]).max() for w in want if np.isfinite(w).any()])
            assert np.abs(a[fin] - b[fin]).max() <= TOL[dtype] * scale, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nan_cost_a_few_times_a_call_at_most(dtype):
    """A value that a row sees, or that is hidden from some rows of a tile, or any number of them: a wave's products
    are formed at most once more for every 32 columns (four here), from memory, where a walk along the keys took a
    hundred times a call. The bound leaves room for both and for the clock."""
    n = 1500
    attn = layers.CrossAttention("128x0e+128x1o", 4, dtype=dtype)
    s = layers.Samples([0, n])
    b = attn.batch(s, s, causal=True)
    rng = np.random.default_rng(53)
    q, k, v, g = (dev(rng.standard_normal((n, 512)), dtype) for _ in range(4))

    def us(f):
        f()
        best = 1e9
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            f()
            end.record()
            torch.cuda.synchronize()
            best = min(best, 1e3 * start.elapsed_time(end))
        return best

    out, lse = attn.forward(b, q, k, v, need_lse=True)
    clean = us(lambda: attn.forward(b, q, k, v)), us(lambda: attn.backward(b, q, k, v, out, lse, g))
    for rows, bad in ((slice(3, 4), float("nan")), (slice(n - 20, n - 19), float("nan")), (slice(0, n), float("nan")),
                      (slice(0, n), float("inf"))):
        x = v.clone()
        x[rows] = bad
        o, l = attn.forward(b, q, k, x, need_lse=True)
        got = us(lambda: attn.forward(b, q, k, x)), us(lambda: attn.backward(b, q, k, x, o, l, g))
        y = g.clone()
        y[rows] = bad
        got += (us(lambda: attn.backward(b, q, k, v, out, lse, y)),)
        print("us", dtype, rows, bad, "clean", clean, "got", got, flush=True)
        assert got[0] <= 16 * clean[0] and max(got[1:]) <= 16 * clean[1]


def refused_fast(make):
    """The call is refused as unsupported, without lists laid out for it before: 67 million tiles take half a
    second and half a gigabyte, a refusal some microseconds."""
    import time
    best = 1e9
    for _ in range(3):
        start = time.perf_counter()
        with pytest.raises(cgtp.CgtpError) as e:
            make()
        best = min(best, time.perf_counter() - start)
        assert e.value.status == 3
    assert best < 0.02, best


@pytest.mark.parametrize("kv_heads", [1, 4])
def test_more_shared_rows_than_one_launch_packs_are_refused_before_they_are_laid_out(kv_heads):
    attn = layers.CrossAttention("32x0e", 4, kv_heads=kv_heads, dtype="bf16")
    tiles = ((1 << 24) - 1) // kv_heads // 8 * 8                 # the packing rounds up to eight
    s = layers.Samples([0, 1])
    for shared in (32 * tiles + 1, (1 << 31) - 200):
        refused_fast(lambda: attn.cache(2, 4, shared=shared))
        refused_fast(lambda: attn.batch(s, s, shared=shared))


def test_the_largest_caches_by_their_tiles():
    """With 64 heads on one context head a slot has two tiles of query rows."""
    attn = layers.CrossAttention("64x0e", 64, kv_heads=1, dtype="bf16")
    for slots, capacity in (((1 << 23), 1), (1 << 10, (1 << 24) + 1)):
        refused_fast(lambda: attn.cache(slots, capacity))
    refused_fast(lambda: attn.cache(1, (1 << 30) + 1))
    h = layers._vp()
    # (the handle alone: no caches of that size)
    status = layers._lib.cgtp_attn_cache_create(attn._h, 1 << 10, 1 << 24, 0, layers.ctypes.byref(h))
    assert status == 0 and layers._lib.cgtp_attn_cache_destroy(h) == 0
