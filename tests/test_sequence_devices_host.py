"""Host-side checks of where a cache and the tensors of its calls lie (CPU only): what is on
another device than the cache is refused before the library is called."""

import pytest

torch = pytest.importorskip("torch")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")


class Tensor:
    """Stands for a tensor on device `index` (-1: the host)."""

    def __init__(self, shape, dtype=torch.float32, index=0):
        self.shape, self.dtype, self.index, self.is_cuda = torch.Size(shape), dtype, index, index >= 0
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def element_size(self):
        return 4


class Library:
    """Every entry point succeeds, and notes that it was called."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        def call(*args):
            self.called.append(name)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(layers, "_lib", lib)
    monkeypatch.setattr(layers, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return lib


def made(shared=0):
    attn = layers.CrossAttention.__new__(layers.CrossAttention)
    attn.heads = attn.kv_heads = 4
    attn.dim_q = attn.dim_kv = 32
    attn.scale, attn._dtype, attn._h = 1.0, torch.float32, None
    cache = layers.AttentionCache.__new__(layers.AttentionCache)
    cache.attn, cache.slots, cache.capacity, cache.shared, cache._index = attn, 2, 8, shared, 0
    cache._h, cache._context_bytes, cache.workspace_size = None, 64, 0
    cache.k, cache.v = Tensor((2, 8, 32)), Tensor((2, 8, 32))
    cache._context = Tensor((64,), torch.uint8) if shared else None
    return attn, cache


def arguments():
    return dict(q=Tensor((2, 32)), k=Tensor((2, 32)), v=Tensor((2, 32)), lengths=Tensor((2,), torch.int32),
                out=Tensor((2, 32)), lse=Tensor((2, 4)), ws=Tensor((64,), torch.uint8))


@pytest.mark.parametrize("device", ["cpu", "cuda:1", "cuda:7", "meta"])
def test_a_cache_lies_on_the_current_device(library, device):
    attn, _ = made()
    with pytest.raises(ValueError):
        layers.AttentionCache(attn, 2, 8, device=device)
    assert library.called == []


@pytest.mark.parametrize("name", ["q", "k", "v", "lengths", "out", "lse", "ws"])
@pytest.mark.parametrize("index", [-1, 1])
def test_a_step_refuses_tensors_of_another_device(library, name, index):
    attn, cache = made()
    args = arguments()
    attn.step(cache, **args)
    assert library.called == ["cgtp_attn_step"]
    args[name] = Tensor(args[name].shape, args[name].dtype, index)
    with pytest.raises(ValueError):
        attn.step(cache, **args)
    assert library.called == ["cgtp_attn_step"]


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("index", [-1, 1])
def test_caches_moved_to_another_device_are_refused(library, name, index):
    attn, cache = made(shared=3)
    setattr(cache, name, Tensor((2, 8, 32), index=index))
    with pytest.raises(ValueError):
        attn.step(cache, **arguments())
    if name == "k":
        with pytest.raises(ValueError):
            cache.share(Tensor((3, 32)), Tensor((3, 32)))
    assert library.called == []


@pytest.mark.parametrize("name", ["k", "v", "key_mask"])
@pytest.mark.parametrize("index", [-1, 1])
def test_shared_rows_of_another_device_are_refused(library, name, index):
    _, cache = made(shared=3)
    args = dict(k=Tensor((3, 32)), v=Tensor((3, 32)), key_mask=Tensor((3,), torch.bool))
    cache.share(**args)
    assert library.called == ["cgtp_attn_cache_share"]
    args[name] = Tensor(args[name].shape, args[name].dtype, index)
    with pytest.raises(ValueError):
        cache.share(**args)
    assert library.called == ["cgtp_attn_cache_share"]
