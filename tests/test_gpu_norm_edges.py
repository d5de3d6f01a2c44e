"""GPU group norm at the edges of its range: empty samples beside others, the
kernels of long samples in every type and lane width, limits of its arguments."""

import numpy as np
import pytest

from oracle import layers as ol
from tests.gpu_util import TOL, assert_close, dev, host, rel_err
from tests.test_gpu_norm import EPS, block_cols, check, inputs, ptr_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("irreps,lens", [("8x0e+4x1o+4x2e", [0, 3, 0, 40, 0]),              # one launch a direction
                                         ("32x0e+32x1o", [0, 1500, 0, 3, 0])])              # runs
def test_statistics_of_empty_samples_are_not_used(irreps, lens, dtype):
    """The forward leaves them as they were: NaN or infinite in reused memory."""
    x, w, b, g = inputs(irreps, lens, dtype)
    ptr = ptr_of(lens)
    sm, norm = layers.Samples(ptr), layers.GroupNorm(irreps, 2, activation="silu", eps=EPS, dtype=dtype)
    args = (irreps, 2, ptr, host(x), host(w), host(b), EPS, "silu")
    ref = ol.norm_backward(*args, host(g))
    for fill in (float("nan"), float("inf"), -float("inf")):
        stats = torch.full((sm.S, norm.num_groups, 2), fill, device="cuda",
                           dtype=torch.float64 if dtype == "f64" else torch.float32)
        y, stats = norm.forward(sm, x, w, b, stats=stats)
        gx, gw, gb = norm.backward(sm, x, w, b, stats, g)
        torch.cuda.synchronize()
        assert_close(host(y), ol.norm_forward(*args), block_cols(irreps), dtype, "y")
        assert_close(host(gx), ref[0], block_cols(irreps), dtype, "grad_x")
        assert rel_err(host(gw), ref[1]) <= TOL[dtype] and rel_err(host(gb), ref[2]) <= TOL[dtype]


@pytest.mark.parametrize("dtype,eps", [("f32", 1.2e-38), ("bf16", 1.2e-38), ("f64", 2.3e-308)])
def test_smallest_eps_leaves_constant_groups_finite(dtype, eps):
    norm, sm = layers.GroupNorm("8x0e+8x1o", 2, activation="silu", eps=eps, dtype=dtype), layers.Samples([0, 4])
    x = torch.zeros((4, norm.dim), dtype=norm.torch_dtype, device="cuda")
    x[:, :8] = 3
    y, stats = norm.forward(sm, x)
    gx = norm.backward(sm, x, None, None, stats, torch.zeros_like(x), need=(True, False, False))[0]
    torch.cuda.synchronize()
    assert torch.all(y == 0) and torch.all(gx == 0)


def test_more_workgroups_than_one_launch_holds():
    """1.1 million samples of one row (every 1000th empty) and 16 blocks: more than 2^24
    sample-strips, where a launch of 256 threads a workgroup ends. Against the formula
    in torch's 64 bits, block by block.

    x is at most 6 and a group of eight has a deviation of 1/15 at least, so its mean's
    three roundings are 15 * 3 * 2^-24 * 6 = 2e-5 of y and 1e-3 of grad_x at most, 1e-5 and
    1e-4 of the largest; a parameter's sum adds 16 rows of 7 * 10^4 terms in sequence,
    each rounded to 2^-24 of a partial sum."""
    S, blocks = 1_100_000, 8
    irreps = "+".join(["8x0e+8x1o"] * blocks)
    lens = np.ones(S, np.int64)
    lens[::1000] = 0
    sm, norm = layers.Samples(ptr_of(lens)), layers.GroupNorm(irreps, 1, activation="none", eps=EPS)
    rows = int(lens.sum())
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, g = (torch.randn((rows, norm.dim), generator=gen, device="cuda") for _ in range(2))
    w = torch.linspace(0.5, 1.5, norm.channels, device="cuda")
    b = torch.linspace(-1, 1, norm.biases, device="cuda")
    y, stats = norm.forward(sm, x, w, b)
    gx, gw, gb = norm.backward(sm, x, w, b, stats, g)
    for i in range(2 * blocks):
        m, even = (1, True) if i % 2 == 0 else (3, False)
        off = i // 2 * 32 + (0 if even else 8)
        cols = slice(off, off + 8 * m)
        xb, gb_ = (t[:, cols].double().view(rows, m, 8) for t in (x, g))
        wi = w[8 * i:8 * i + 8].double()
        xc = xb - xb.mean((1, 2), keepdim=True) if even else xb
        r = (xc.square().mean((1, 2), keepdim=True) + EPS) ** -0.5
        xh, gh = xc * r, gb_ * wi
        want = xh * wi
        d = gh - xh * (gh * xh).mean((1, 2), keepdim=True)
        if even:
            want = want + b[4 * i:4 * i + 8].double()
            d = d - gh.mean((1, 2), keepdim=True)
            sums = gb_.sum((0, 1))
            assert (gb[4 * i:4 * i + 8].double() - sums).abs().max() <= 1e-5 * gb_.abs().sum((0, 1)).max()
        assert (y[:, cols].double().view(rows, m, 8) - want).abs().max() <= 1e-5 * want.abs().max()
        want = d * r
        assert (gx[:, cols].double().view(rows, m, 8) - want).abs().max() <= 1e-4 * want.abs().max()
        sums = (gb_ * xh).sum((0, 1))
        assert (gw[8 * i:8 * i + 8].double() - sums).abs().max() <= 1e-5 * (gb_ * xh).abs().sum((0, 1)).max()


def test_more_runs_than_one_launch_holds():
    """17 million samples of one row and one of 70,000 rows, a row holding one element: more
    than 2^24 runs in one slice. A lone odd scalar gives y = x w / sqrt(x^2 + eps)
    and grad_x = g w eps / (x^2 + eps)^(3/2): the difference of two terms g w / sqrt(x^2 + eps),
    each of some eight roundings of 2^-24."""
    S = 17_000_001
    lens = np.ones(S, np.int64)
    lens[S // 2] = 70_000
    sm, norm = layers.Samples(ptr_of(lens)), layers.GroupNorm("1x0o", 1, eps=EPS)
    assert norm.workspace_size(sm) > 0
    rows = int(lens.sum())
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, g = (torch.randn((rows, 1), generator=gen, device="cuda") for _ in range(2))
    w = torch.full((1,), 1.25, device="cuda")
    y, stats = norm.forward(sm, x, w)
    gx, gw, _ = norm.backward(sm, x, w, None, stats, g, need=(True, True, False))
    xd, gd = x.double(), 1.25 * g.double()
    var, lo, hi = xd * xd, S // 2, S // 2 + 70_000
    var[lo:hi] = var[lo:hi].mean()
    r = (var + EPS) ** -0.5
    xh = xd * r
    along = gd * xh
    along[lo:hi] = along[lo:hi].mean()
    assert ((y - 1.25 * xh).abs() <= 1e-6 * (1.25 * xh).abs()).all()
    assert ((gx - (gd - xh * along) * r).abs() <= 2e-6 * (gd.abs() + (xh * along).abs()) * r).all()
    total = (g * xh).sum()
    assert abs(gw.double().item() - total.item()) <= 1e-5 * (g * xh).abs().sum().item()


# (irreps, groups, activation, lengths): the longest sample's part of a narrow strip exceeds 256 KB in every type
RUNS = [
    ("32x0e+32x1o", 4, "silu", [2800, 3]),
    ("35x0e+21x1o+7x2e", 7, "gelu", [0, 4700, 0, 5, 5100, 0]),           # single-channel lanes in fp32 and bf16
    ("16x0e+8x0o+8x3o+8x4e", 4, "gelu", [40, 5000]),                     # 7 and 9 components
    ("1200x0e+300x1o", 1, "none", [150, 0, 400]),                        # groups wider than 256 lanes
    ("8x0e", 2, "silu", [0, 17000, 1]),                                  # more rows than one span of 4096
    ("64x0e+24x0o+8x1e", 2, "silu", [2500, 2500, 1, 900]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("irreps,groups,act,lens", RUNS)
def test_runs_of_rows(irreps, groups, act, lens, dtype):
    norm = layers.GroupNorm(irreps, groups, activation=act, eps=EPS, dtype=dtype)
    assert norm.workspace_size(layers.Samples(ptr_of(lens))) > 0
    x, w, b, g = inputs(irreps, lens, dtype)
    a = check(irreps, groups, act, lens, dtype, x, w, b, g, norm)
    # statistics of empty samples are not written
    again = check(irreps, groups, act, lens, dtype, x, w, b, g, norm)
    assert all(torch.equal(u, v) for u, v in zip(a[:1] + a[2:], again[:1] + again[2:]))

    def shifted(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    check(irreps, groups, act, lens, dtype, shifted(x), shifted(w), shifted(b), shifted(g), norm)


def test_runs_in_a_graph():
    irreps, lens = "32x0e+32x1o+32x2e", [0, 2800, 9]
    x, w, b, g = inputs(irreps, lens, "f32")
    sm, norm = layers.Samples(ptr_of(lens)), layers.GroupNorm(irreps, 4, activation="silu")
    assert norm.workspace_size(sm) > 0

    def step(x):
        y, stats = norm.forward(sm, x, w, b)
        return (y,) + norm.backward(sm, x, w, b, stats, g)

    step(x)
    torch.cuda.synchronize()
    graph, xs = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        res = step(xs)
    for k in range(3):
        xs.copy_(x * (k + 1) + k)
        graph.replay()
        want = step(xs)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(res, want))


def test_more_rows_than_one_slice():
    """430 MB of rows, worked off in slices of at most 160 MB (forward) and 80 MB
    (backward, two tensors): picked samples and the weights' gradients against the
    oracle's formulas in torch's 64 bits."""
    irreps, groups, lens = "128x0e+128x1o", 8, [9000, 0, 70000, 1, 60000, 64000, 0, 7000]
    ptr = ptr_of(lens)
    norm, sm = layers.GroupNorm(irreps, groups, activation="silu", eps=EPS), layers.Samples(ptr)
    assert norm.workspace_size(sm) > 0
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, g = (torch.randn((int(ptr[-1]), norm.dim), generator=gen, device="cuda") for _ in range(2))
    w = torch.linspace(0.5, 1.5, norm.channels, device="cuda")
    b = torch.linspace(-1, 1, norm.biases, device="cuda")
    y, stats = norm.forward(sm, x, w, b)
    gx, gw, gb = norm.backward(sm, x, w, b, stats, g)
    rw, rb = (torch.zeros(n, dtype=torch.float64, device="cuda") for n in (norm.channels, norm.biases))
    for lo, hi in zip(ptr[:-1], ptr[1:]):
        if lo == hi:
            continue
        for m, off, ch in ((1, 0, 0), (3, 128, 128)):
            cols = slice(off, off + 128 * m)
            xb, gy = (t[lo:hi, cols].double().view(-1, m, groups, 16) for t in (x, g))
            xc = xb - xb.mean((0, 1, 3), keepdim=True) if m == 1 else xb
            r = (xc.square().mean((0, 1, 3), keepdim=True) + EPS) ** -0.5
            xh, wb = xc * r, w[ch:ch + 128].double().view(groups, 16)
            z, gz = xh * wb, gy
            if m == 1:
                z = z + b.double().view(groups, 16)
                s = torch.sigmoid(z)
                z, gz = z * s, gy * (s + z * s * (1 - s))
                rb += gz.sum((0, 1)).view(-1)
            rw[ch:ch + 128] += (gz * xh).sum((0, 1)).view(-1)
            gh = gz * wb
            d = gh - xh * (gh * xh).mean((0, 1, 3), keepdim=True)
            if m == 1:
                d = d - gh.mean((0, 1, 3), keepdim=True)
            for got, want in ((y, z), (gx, d * r)):
                want = want.reshape(-1, 128 * m)
                assert (got[lo:hi, cols] - want).abs().max() <= TOL["f32"] * want.abs().max()
    assert (gw - rw).abs().max() <= TOL["f32"] * rw.abs().max()
    assert (gb - rb).abs().max() <= TOL["f32"] * rb.abs().max()


@pytest.mark.parametrize("irreps,act,lens,runs", [("2x0e+1x1o", "silu", [9000, 3], False),     # one workgroup a sample
                                                  ("2x0e+1x1e", "none", [2_200_000, 5], True)])
def test_more_rows_than_one_span(irreps, act, lens, runs):
    """A workgroup walks 4096 rows at a time; narrow rows give it more (a run is a 512th of its sample)."""
    norm = layers.GroupNorm(irreps, 1, activation=act, eps=EPS)
    assert (norm.workspace_size(layers.Samples(ptr_of(lens))) > 0) == runs
    x, w, b, g = inputs(irreps, lens, "f32")
    check(irreps, 1, act, lens, "f32", x, w, b, g, norm)
