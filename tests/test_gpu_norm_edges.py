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
