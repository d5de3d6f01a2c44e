"""GPU group norm with activation against the fp64 oracle: ragged and empty
samples, odd channel counts, groups wider than a workgroup's lanes, misaligned
tensors, missing weights, degenerate statistics, every dtype; gradients also
against differences (fp64); streams, graph capture, refusals."""

import numpy as np
import pytest

from oracle import layers as ol
from oracle.irreps import dim, parse_irreps
from tests.gpu_util import TOL, assert_close, dev, host, rel_err, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

EPS = 1e-5
CASES = [
    ("8x0e+4x1o", 2, "silu", [3, 0, 1, 40]),
    ("5x0e+3x1o+7x2e", 1, "gelu", [2, 33, 65]),
    ("35x0e+21x1o+7x2e", 7, "silu", [0, 70, 5]),
    ("128x0e+128x1o+128x2e", 8, "silu", [21, 9, 130]),
    ("16x0e+16x0o+8x3o+8x4e", 4, "gelu", [50]),
    ("1200x0e+300x1o", 1, "none", [7, 20]),      # a group wider than 256 lanes
    ("512x0e", 256, "silu", [11]),               # more groups than channels in a 16-byte access
    ("4x0e", 4, "none", [1]),                    # one element a group: var = 0
    ("32x0e+32x1o", 4, "silu", [700, 3]),        # several runs a sample
]


def inputs(irreps, lens, dtype, seed=0, shift=0.5):
    rng = np.random.default_rng(seed)
    n, d = sum(lens), dim(parse_irreps(irreps))
    bl = ol.blocks(irreps)
    c, b = sum(x[0] for x in bl), sum(x[0] for x in bl if x[5] is not None)
    x = rng.standard_normal((n, d)) * 1.5
    for mul, l, p, off, _, bias in bl:
        if bias is not None:
            x[:, off:off + mul] += shift
    return [dev(a, dtype) for a in (x, 1 + 0.3 * rng.standard_normal(c), 0.3 * rng.standard_normal(b),
                                    rng.standard_normal((n, d)))]


def block_cols(irreps):
    return [(off, mul * (2 * l + 1)) for mul, l, _, off, _, _ in ol.blocks(irreps)]


def ptr_of(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def check(irreps, groups, act, lens, dtype, x, w, b, g, norm=None):
    ptr = ptr_of(lens)
    sm = layers.Samples(ptr)
    norm = norm or layers.GroupNorm(irreps, groups, activation=act, eps=EPS, dtype=dtype)
    y, stats = norm.forward(sm, x, w, b)
    gx, gw, gb = norm.backward(sm, x, w, b, stats, g)
    torch.cuda.synchronize()
    hx, hw, hb, hg = host(x), host(w), host(b), host(g)
    assert_close(host(y), ol.norm_forward(irreps, groups, ptr, hx, hw, hb, EPS, act), block_cols(irreps), dtype, "y")
    rx, rw, rb = ol.norm_backward(irreps, groups, ptr, hx, hw, hb, EPS, act, hg)
    # a one-element group's gradient is what rounding leaves of a zero: judged against the size of g / sqrt(eps)
    lone = sum(lens) == 1 and groups == ol.blocks(irreps)[0][0]
    if lone:
        assert np.abs(host(gx)).max() <= TOL[dtype] * np.abs(hg).max() / np.sqrt(EPS)
    else:
        assert_close(host(gx), rx, block_cols(irreps), dtype, "grad_x")
    if not lone:
        assert rel_err(host(gw), rw) <= TOL[dtype]
    assert rel_err(host(gb), rb) <= TOL[dtype]
    return y, stats, gx, gw, gb


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("irreps,groups,act,lens", CASES)
def test_norm(irreps, groups, act, lens, dtype):
    x, w, b, g = inputs(irreps, lens, dtype)
    check(irreps, groups, act, lens, dtype, x, w, b, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_misaligned_and_repeatable(dtype):
    irreps, lens = "32x0e+16x1o", [5, 60]
    x, w, b, g = inputs(irreps, lens, dtype)

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return s.copy_(t)

    a = check(irreps, 4, "silu", lens, dtype, x, w, b, g)
    a2 = check(irreps, 4, "silu", lens, dtype, x, w, b, g)
    assert all(torch.equal(u, v) for u, v in zip(a, a2))
    check(irreps, 4, "silu", lens, dtype, shifted(x), shifted(w), shifted(b), shifted(g))


def test_norm_large_mean_keeps_its_variance():
    # fp32 inputs about 100 with deviation 1.5: a difference of squares would lose 1e4 * 6e-8 of
    # the variance; sums about a pivot keep the framework's 1e-5 (the mean itself rounds to 4e-6)
    irreps, lens = "32x0e", [400]
    x, w, b, g = inputs(irreps, lens, "f32", shift=100.0)
    check(irreps, 4, "none", lens, "f32", x, w, b, g)


def test_norm_constant_rows_and_no_weights():
    irreps, ptr = "8x0e+8x1o", [0, 4]
    norm = layers.GroupNorm(irreps, 2, activation="silu", eps=EPS)
    x = torch.full((4, norm.dim), 3.0, device="cuda")
    x[:, 8:] = 0
    y, stats = norm.forward(layers.Samples(ptr), x)
    g = torch.ones_like(x)
    gx, gw, gb = norm.backward(layers.Samples(ptr), x, None, None, stats, g, need=(True, False, False))
    torch.cuda.synchronize()
    assert gw is None and gb is None
    assert torch.all(y == 0) and torch.isfinite(gx).all()


def test_norm_gradients_match_differences():
    irreps, groups, lens = "4x0e+2x0o+6x1o", 2, [3, 17]
    x, w, b, g = inputs(irreps, lens, "f64", seed=4)
    sm = layers.Samples(ptr_of(lens))
    norm = layers.GroupNorm(irreps, groups, activation="gelu", eps=EPS, dtype="f64")
    f = lambda *a: (norm.forward(sm, *a)[0] * g).sum().item()
    grads = norm.backward(sm, x, w, b, norm.forward(sm, x, w, b)[1], g)
    for k in range(3):
        args = [x, w, b]
        d = dev(np.random.default_rng(30 + k).standard_normal(args[k].shape), "f64")
        h = 1e-6
        up, dn = list(args), list(args)
        up[k], dn[k] = args[k] + h * d, args[k] - h * d
        num = (f(*up) - f(*dn)) / (2 * h)
        assert abs(num - (grads[k] * d).sum().item()) < 1e-6 * (1 + abs(num))


def test_norm_empty_batches():
    norm = layers.GroupNorm("8x0e+8x1o", 2, activation="silu")
    w, b = torch.ones(norm.channels, device="cuda"), torch.zeros(norm.biases, device="cuda")
    for ptr in ([0], [0, 0, 0]):
        sm = layers.Samples(ptr)
        x = torch.empty((0, norm.dim), device="cuda")
        y, stats = norm.forward(sm, x, w, b)
        gx, gw, gb = norm.backward(sm, x, w, b, stats, x)
        torch.cuda.synchronize()
        assert y.shape == x.shape == gx.shape
        assert torch.all(gw == 0) and torch.all(gb == 0)


def test_norm_nan_stays_in_its_sample():
    irreps, lens = "8x0e+8x1o", [40, 40]
    x, w, b, _ = inputs(irreps, lens, "f32")
    norm = layers.GroupNorm(irreps, 2, activation="silu")
    sm = layers.Samples(ptr_of(lens))
    clean, _ = norm.forward(sm, x, w, b)
    x2 = x.clone()
    x2[3, 0] = float("nan")
    y, _ = norm.forward(sm, x2, w, b)
    torch.cuda.synchronize()
    assert torch.isnan(y[:40, :4]).all()
    assert torch.equal(y[40:], clean[40:]) and torch.equal(y[:40, 4:], clean[:40, 4:])


def test_norm_on_a_side_stream_and_in_a_graph():
    irreps, lens = "32x0e+32x1o+32x2e", [9, 21, 300]
    x, w, b, g = inputs(irreps, lens, "f32")
    sm = layers.Samples(ptr_of(lens))
    norm = layers.GroupNorm(irreps, 4, activation="silu")
    y0, st0 = norm.forward(sm, x, w, b)
    want = (y0, *norm.backward(sm, x, w, b, st0, g))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, st = norm.forward(sm, x, w, b)
        got = (y, *norm.backward(sm, x, w, b, st, g))
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        yg, stg = norm.forward(sm, xs, w, b)
        gg = norm.backward(sm, xs, w, b, stg, g)
    for k in range(3):
        xs.copy_(x * (k + 1) + k)
        graph.replay()
        e, es = norm.forward(sm, xs, w, b)
        eg = norm.backward(sm, xs, w, b, es, g)
        torch.cuda.synchronize()
        assert torch.equal(yg, e) and all(torch.equal(u, v) for u, v in zip(gg, eg))


def test_norm_refusals():
    norm = layers.GroupNorm("8x0e+8x1o", 2)
    sm = layers.Samples([0, 4])
    x = torch.zeros((4, norm.dim), device="cuda")
    y, stats = norm.forward(sm, x)
    with pytest.raises(ValueError):
        norm.forward(sm, x[:3])
    with pytest.raises(ValueError):
        norm.forward(sm, x.half())
    with pytest.raises(ValueError):
        norm.forward(sm, x, weight=torch.ones(3, device="cuda"))
    with pytest.raises(cgtp.CgtpError) as e:
        norm.backward(sm, x, None, None, stats, x, ws=torch.empty(4, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    ws = torch.empty(norm.workspace_size(sm, backward=True) + 16, dtype=torch.uint8, device="cuda")[1:]
    with pytest.raises(cgtp.CgtpError) as e:
        norm.backward(sm, x, None, None, stats, x, ws=ws)
    assert e.value.status == 1
