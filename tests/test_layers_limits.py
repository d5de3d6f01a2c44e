"""Host-side limits of the layers (CPU only): values that the kernels' types do
not hold."""

import pytest

cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")


@pytest.mark.parametrize("dtype,bad", [("f32", (1e-50, 1e-39, 1e39)), ("bf16", (1e-50, 1e-39, 1e39)),
                                       ("f64", (5e-324, 1e-310))])
def test_eps_has_to_be_a_normal_number_of_the_arithmetic(dtype, bad):
    """As 0 in 32 bits it would leave 0 * inf = NaN where a group's variance is zero."""
    for eps in bad:
        with pytest.raises(cgtp.CgtpError) as e:
            layers.GroupNorm("8x0e", 2, eps=eps, dtype=dtype)
        assert e.value.status == 1 and "eps" in str(e.value)
