"""Host-side limits of the layers (CPU only): values that the kernels' types do
not hold, and a handle that threads share."""

import gc
import weakref

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


class Layout:
    """Stands for a Samples object: its handle is the number that the library is asked about."""

    def __init__(self, handle):
        self._h = handle


def bare_norm(monkeypatch, cls=layers.GroupNorm):
    def size(norm, samples, backward, out):
        out._obj.value = 100 * samples + backward
        return 0

    monkeypatch.setattr(layers, "_lib", type("Lib", (), {"cgtp_norm_workspace_size": staticmethod(size)}))
    return cls.__new__(cls)


def test_workspace_size_is_the_layouts_own_whatever_another_thread_asks(monkeypatch):
    """Another thread's call is put after each attribute that the first one's sets, where
    a switch of threads may fall."""
    other = Layout(2)

    class Switched(layers.GroupNorm):
        busy = False

        def __setattr__(self, name, value):
            object.__setattr__(self, name, value)
            if name.startswith("_siz") and not Switched.busy:
                Switched.busy = True
                assert self.workspace_size(other, backward=True) == 201
                Switched.busy = False

    norm = bare_norm(monkeypatch, Switched)
    norm.__dict__["_sized"] = None
    one = Layout(1)
    for backward in (False, True, False):
        assert norm.workspace_size(one, backward=backward) == 100 + backward
    assert norm.workspace_size(other) == 200


def test_a_norm_does_not_keep_the_last_layout(monkeypatch):
    norm = bare_norm(monkeypatch)
    norm._sized = None
    one = Layout(1)
    assert norm.workspace_size(one) == 100
    ref = weakref.ref(one)
    del one
    gc.collect()
    assert ref() is None
    assert norm.workspace_size(Layout(3)) == 300
