"""The example block (linear maps, group norm, attention, dropout) as a whole:
outputs and every gradient against the same composition of fp64 oracles, and the
training loop's loss."""

import numpy as np
import pytest

from oracle import layers as ol
from oracle import linear as olin
from tests.gpu_util import dev, host, rel_err

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
context_block = pytest.importorskip("examples.context_block")

# Five stages forward and five backward; each adds at most 1e-5 (fp32 sums) or the
# half unit 2^-9 that its stored bf16 results are rounded by, of the largest
# element, and passes an input's error on about unchanged (weights of variance
# 1 / inputs, rows normed to size one, scores of size one). A factor of two for
# attention weights and score gradients, which bf16 also rounds.
TOL = {"f32": 10 * 2 * 1e-5, "bf16": 10 * 2 * 2.0 ** -9}

CASES = [
    ("32x0e+32x1o+32x2e", "16x0e+16x1o+16x2e", 4, 2, 4, [21, 9, 21], [40, 0, 33], False),
    ("35x0e+21x1o+7x2e", "10x0e+6x1o", 7, 1, 7, [1, 70], [65, 3], True),       # no path feeds k's degree 2
    ("64x0e+64x1o", "24x0e+8x1o+8x0e", 2, 2, 8, [130], [200], True),           # two scalar blocks feed one
]


def oracle_block(block, irreps, context, heads, kv_heads, groups, nptr, cptr, x, c, mask, w, step, g):
    """(y, {name: gradient}) in fp64 from the device's own inputs."""
    kv = ol.kv_irreps(irreps, heads, kv_heads)
    Lq, Lkv = olin.LinearLayout(irreps, irreps), olin.LinearLayout(context, kv + "+" + kv)
    dk = Lkv.dim_out // 2
    n = ol.norm_forward(irreps, groups, nptr, x, w["norm_w"], w["norm_b"], 1e-5, "silu")
    q, t = olin.forward(Lq, n, w["w_q"]), olin.forward(Lkv, c, w["w_kv"])
    k, v = t[:, :dk], t[:, dk:]
    a = ol.attn_forward(irreps, heads, kv_heads, nptr, cptr, q, k, v, mask, block.attn.scale)[0]
    keep, gain = ol.dropout_mask(irreps, range(x.shape[0]), block.p, block.seed, step)
    drop = keep * gain
    y = x + drop * olin.forward(Lq, a, w["w_out"])
    r = {}
    ga, r["w_out"] = olin.backward(Lq, a, w["w_out"], drop * g)
    gq, gk, gv = ol.attn_backward(irreps, heads, kv_heads, nptr, cptr, q, k, v, mask, block.attn.scale, ga)
    r["c"], r["w_kv"] = olin.backward(Lkv, c, w["w_kv"], np.concatenate([gk, gv], 1))
    gn, r["w_q"] = olin.backward(Lq, n, w["w_q"], gq)
    gx, r["norm_w"], r["norm_b"] = ol.norm_backward(irreps, groups, nptr, x, w["norm_w"], w["norm_b"], 1e-5, "silu", gn)
    r["x"] = gx + g
    return y, r


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("irreps,context,heads,kv_heads,groups,nq,nk,masked", CASES)
def test_context_block(irreps, context, heads, kv_heads, groups, nq, nk, masked, dtype):
    nptr, cptr = (np.concatenate([[0], np.cumsum(n)]) for n in (nq, nk))
    block = context_block.ContextBlock(irreps, context, heads, kv_heads, groups, p=0.25, dtype=dtype, seed=5)
    rng = np.random.default_rng(11)
    x = dev(rng.standard_normal((nptr[-1], block.norm.dim)), dtype)
    c = dev(rng.standard_normal((cptr[-1], block.to_kv.dim_in)), dtype)
    g = dev(rng.standard_normal(tuple(x.shape)), dtype)
    block.params["norm_w"].copy_(dev(rng.uniform(0.5, 1.5, block.norm.channels), dtype))
    block.params["norm_b"].copy_(dev(rng.standard_normal(block.norm.biases), dtype))
    mask = torch.from_numpy(rng.random(cptr[-1]) > 0.3).cuda() if masked else None
    y, saved = block.forward(context_block.Layout(block, nptr, cptr), x, c, 3, key_mask=mask)
    gx, gc, grads = block.backward(saved, g)
    torch.cuda.synchronize()
    w = {name: host(p) for name, p in block.params.items()}
    ry, r = oracle_block(block, irreps, context, heads, kv_heads, groups, nptr, cptr, host(x), host(c),
                         None if mask is None else mask.cpu().numpy(), w, 3, host(g))
    grads = dict(grads, x=gx, c=gc)
    assert rel_err(host(y), ry) <= TOL[dtype]
    assert set(grads) == set(r)
    for name in r:
        err = rel_err(host(grads[name]), r[name])
        assert err <= TOL[dtype], "%s: %.3e" % (name, err)


def test_training_lowers_the_loss(capsys):
    losses = context_block.main(steps=40)
    assert np.isfinite(losses).all() and losses[-1] < 0.7 * losses[0]
    assert "step  39" in capsys.readouterr().out
