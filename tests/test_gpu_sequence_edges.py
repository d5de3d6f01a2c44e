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
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("seen", SEEN)
def test_few_rows_whose_parts_see_no_shared_key(seen, causal, dtype):
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
    out, lse = attn.forward(batch, q, k, v, scale=1.0, key_mask=mask, need_lse=True)
    torch.cuda.synchronize()
    hm = mask.cpu().numpy()
    ro, rl = ol.seq_forward("128x0e", heads, heads, qp, kp, host(q), host(k), host(v), hm, 1.0, causal, shared)
    assert np.isfinite(host(out)).all() and np.isfinite(host(lse)).all()
    assert rl.max() < -150.0
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
