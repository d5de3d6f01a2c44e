"""GPU dropout against the oracle's generator: the mask bit for bit, values,
residual, backward, odd channel counts, misaligned tensors, refusals."""

import numpy as np
import pytest

from oracle import layers as ol
from oracle.irreps import dim, parse_irreps
from tests.gpu_util import TOL, dev, host, rel_err

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

SEED, OFFSET = 0xFEDCBA9876543210, 0xDEADBEEF


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f64"])
@pytest.mark.parametrize("irreps,rows", [("8x0e", 1), ("32x0e+32x1o+32x2e", 70), ("35x0e+21x1o+7x2e", 33),
                                         ("1x0e+3x3o+2x4e", 300), ("2100x0e", 5), ("128x0e+128x1o+128x2e+128x3o", 40)])
def test_dropout(irreps, rows, dtype):
    rng = np.random.default_rng(rows)
    d = dim(parse_irreps(irreps))
    x, res, g = (dev(rng.uniform(0.5, 2.0, (rows, d)), dtype) for _ in range(3))
    drop = layers.Dropout(irreps, dtype=dtype)
    for p in (0.0, 0.3, 0.999999):
        keep, scale = ol.dropout_mask(irreps, range(rows), p, SEED, OFFSET)
        y = drop.forward(x, p, SEED, OFFSET)
        gx = drop.backward(g, p, SEED, OFFSET)
        yr = drop.forward(x, p, SEED, OFFSET, residual=res)
        inplace = drop.forward(x, p, SEED, OFFSET, residual=res, out=res.clone())
        torch.cuda.synchronize()
        assert np.array_equal(host(y) != 0, keep) and np.array_equal(host(gx) != 0, keep)
        assert rel_err(host(y), keep * host(x) * scale) <= TOL[dtype]
        assert rel_err(host(gx), keep * host(g) * scale) <= TOL[dtype]
        assert rel_err(host(yr), host(res) + keep * host(x) * scale) <= TOL[dtype]
        assert torch.equal(yr, inplace)
        if p == 0.0:
            assert torch.equal(y, x)


def test_dropout_misaligned_matches_aligned():
    drop = layers.Dropout("32x0e+16x1o")
    x = torch.randn((50, drop.dim), device="cuda")
    s = torch.empty(x.numel() + 1, device="cuda")[1:].view(x.shape).copy_(x)
    assert torch.equal(drop.forward(x, 0.4, 3, 1), drop.forward(s, 0.4, 3, 1))


def test_dropout_offsets_differ_and_dropped_nan_is_zero():
    drop = layers.Dropout("64x0e")
    x = torch.full((64, 64), float("nan"), device="cuda")
    a, b = drop.forward(x, 0.5, 3, 1), drop.forward(x, 0.5, 3, 2)
    torch.cuda.synchronize()
    assert torch.all((a == 0) | torch.isnan(a))
    # 4096 fair draws agree in 2048 places, deviation 32; six of them
    same = int((torch.isnan(a) == torch.isnan(b)).sum())
    assert abs(same - 2048) < 200


def test_dropout_empty_and_large_row_counts():
    drop = layers.Dropout("8x0e", dtype="bf16")
    assert drop.forward(torch.empty((0, 8), dtype=torch.bfloat16, device="cuda"), 0.5, 1, 1).shape == (0, 8)
    rows = 3_000_001                    # more rows than one pass of the grid holds
    x = torch.ones((rows, 8), dtype=torch.bfloat16, device="cuda")
    y = drop.forward(x, 0.5, SEED, 5)
    pick = [0, 1, 1 << 20, rows - 1]
    keep, _ = ol.dropout_mask("8x0e", pick, 0.5, SEED, 5)
    torch.cuda.synchronize()
    assert np.array_equal(host(y[pick]) != 0, keep)


def test_dropout_refusals():
    drop = layers.Dropout("8x0e")
    x = torch.ones((4, 8), device="cuda")
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(cgtp.CgtpError) as e:
            drop.forward(x, p, 1, 1)
        assert e.value.status == 1
    with pytest.raises(ValueError):
        drop.forward(x, 0.1, 1 << 64, 1)
    with pytest.raises(ValueError):
        drop.forward(x, 0.1, 1, 1 << 32)
    with pytest.raises(ValueError):
        drop.forward(x, 0.1, 1, 1, residual=x[:2])
    with pytest.raises(ValueError):
        drop.forward(x.t(), 0.1, 1, 1)
