"""GPU single tokens on caches against the fp64 oracle: ragged, empty, full and idle
slots, grouped heads up to more than a tile of them, odd channel counts, head sizes
up to 256, splits, shared rows with masks, strided rows, what lies behind a
sequence's end, graph replays that count on, the run of a prompt and its tokens, refusals."""

import numpy as np
import pytest

from oracle import layers as ol
from oracle.irreps import dim, parse_irreps
from tests.gpu_util import TOL, dev, host, rel_err, torch_dtype
from tests.test_gpu_attention import ptr_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
cgtp = pytest.importorskip("clebsch_gordan_tensor_amd.cgtp")
layers = pytest.importorskip("clebsch_gordan_tensor_amd.layers")

# (irreps, heads, kv heads, lengths, capacity, shared rows)
CASES = [
    ("8x0e", 1, 1, [0], 1, 0),
    ("8x0e", 1, 1, [0, -1, 3], 4, 0),
    ("32x0e+32x1o+32x2e", 4, 4, [5, 31, 32, 63, -1, 64], 64, 0),              # one idle, one full
    ("10x0e+6x1o", 2, 1, [0, 33, 70], 80, 0),                                # element-wise rows
    ("35x0e+21x1o+7x2e", 7, 1, [100, 3], 200, 0),                            # 7 heads share a context head
    ("64x0e", 64, 1, [40, 0, 7], 50, 0),                                     # two tiles of heads
    ("64x0e", 2, 2, [300, 2], 700, 0),
    ("128x0e+128x1o", 4, 2, [700, 90, 127], 1000, 0),                        # heads of 128
    ("128x0e+128x1o+128x2e", 8, 4, [50, 140], 150, 0),                       # 144, padded to 160
    ("96x0e+96x1o+24x2e", 6, 3, [65], 97, 0),                                # 84
    ("24x0e+24x1o+24x2e+24x3o", 2, 1, [33], 50, 0),                          # 192
    ("14x0e+14x1o+14x2e+14x3o", 1, 1, [40], 70, 0),                          # 224
    ("128x0e+128x1o+128x2e+128x3o", 8, 8, [70, 9], 80, 0),                   # 256
    ("128x0e+128x1o+128x2e+128x3o", 16, 4, [1500, 1, 900], 1600, 0),         # splits
    ("128x0e+128x1o+128x2e+128x3o", 16, 16, [200, 33], 256, 0),              # several workgroups of heads
    ("64x0e", 4, 2, [3, -1, 0] * 250 + [900, 127], 1000, 0),                 # more slots than workgroups at once
    ("64x0e", 4, 4, [-1] * 70 + [2000] + [-1] * 10 + [31], 2001, 0),         # one long among idle ones
    ("64x0e", 64, 1, [300, 0, 700, -1, 40], 701, 0),                         # two tiles of heads, shared out
    ("128x0e+128x1o+128x2e+128x3o", 8, 8, [500, 9, 31, 470], 600, 0),        # 256, shared out
    ("35x0e+21x1o+7x2e", 7, 1, [100, 3, 900, 0, 64], 1000, 0),
    ("32x0e+32x1o+32x2e", 8, 2, [100, 3, 500, 0, 64], 600, 0),               # runs of 8 bytes in bf16
    ("64x0e", 4, 2, [0, 130, -1, 7] * 300, 131, 0),                          # lengths added up beforehand
    ("64x0e", 64, 1, [-1, 40, 200] * 100, 201, 30),
    ("64x0e", 4, 2, [-1, -1, 300], 300, 0),                                  # nobody
    ("8x0e", 1, 1, [0], 1, 1),
    ("32x0e+32x1o+32x2e", 4, 2, [5, 0, -1, 30, 40], 40, 50),
    ("35x0e+21x1o+7x2e", 7, 1, [100, 3], 101, 333),
    ("64x0e", 8, 1, list(range(40)), 64, 700),                               # 64 rows a wave against the shared
    ("128x0e+128x1o+128x2e+128x3o", 16, 4, [3, 70], 100, 1000),
    ("128x0e+128x1o+128x2e", 8, 4, [3, 70, 200], 300, 200),                  # fp32: two launches
]


def setup(case, dtype, seed=0, mask=None):
    irreps, heads, kv_heads, lens, cap, shared = case
    rng = np.random.default_rng(seed)
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    S, dq, dk = len(lens), attn.dim_q, attn.dim_kv
    q, k, v = (dev(rng.standard_normal((S, d)), dtype) for d in (dq, dk, dk))
    cache = attn.cache(S, cap, shared=shared)
    cache.k.copy_(dev(rng.standard_normal((S, cap, dk)), dtype))
    cache.v.copy_(dev(rng.standard_normal((S, cap, dk)), dtype))
    common = None
    if shared:
        ks, vs = (dev(rng.standard_normal((shared, dk)), dtype) for _ in range(2))
        cache.share(ks, vs, key_mask=mask)
        common = (host(ks), host(vs), None if mask is None else mask.cpu().numpy())
    return attn, cache, q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), common


def check(case, dtype, attn, cache, q, k, v, lengths, common):
    irreps, heads, kv_heads, lens, cap, shared = case
    want = ol.cache_step(irreps, heads, kv_heads, host(q), host(k), host(v), host(cache.k), host(cache.v), lens,
                         attn.scale, common)
    out, lse = attn.step(cache, q, k, v, lengths, need_lse=True)
    torch.cuda.synchronize()
    assert rel_err(host(out), want[0]) <= TOL[dtype]
    gl, rl = host(lse), want[1]
    assert np.array_equal(np.isinf(gl), np.isinf(rl))
    fin = np.isfinite(rl)
    # as the batches': fp32 sums and logarithms of scores of size 10 at most
    assert fin.sum() == 0 or np.abs(gl[fin] - rl[fin]).max() <= 2e-5
    assert np.array_equal(host(cache.k), want[2]) and np.array_equal(host(cache.v), want[3])
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_step(case, dtype):
    print("step", case, dtype, flush=True)
    state = setup(case, dtype)
    a = check(case, dtype, *state)
    b = check(case, dtype, *state)                    # the same row again
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(a[0], state[0].step(*state[1:6]))      # without the lse


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shared", [0, 40])
def test_what_lies_behind_the_end_is_not_used(dtype, shared):
    case = ("32x0e+16x1o", 4, 2, [0, 5, 31, 32, 70, -1, 90], 90, shared)
    attn, cache, q, k, v, lengths, common = setup(case, dtype)
    want = attn.step(cache, q, k, v, lengths)
    for s, n in enumerate(case[3]):
        cache.k[s, n + 1 if 0 <= n < 90 else 0:] = float("nan")
        cache.v[s, n + 1 if 0 <= n < 90 else 0:] = float("inf")
    before = cache.k.clone()
    got, lse = attn.step(cache, q, k, v, lengths, need_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    assert torch.all(got[5:] == 0) and torch.all(torch.isinf(lse[5:])) and torch.isfinite(lse[:5]).all()
    assert torch.equal(before.view(torch.uint8), cache.k.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_shared_rows(dtype):
    mask = torch.from_numpy(np.random.default_rng(2).random(100) < 0.5).cuda()
    for m in (mask, torch.zeros_like(mask)):
        case = ("32x0e+16x1o", 4, 2, [0, 5, 70], 90, 100)
        check(case, dtype, *setup(case, dtype, mask=m))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_and_misaligned_rows(dtype):
    case = ("32x0e+16x1o", 4, 4, [0, 5, 70], 90, 33)
    attn, cache, q, k, v, lengths, common = setup(case, dtype)
    want = attn.step(cache, q, k, v, lengths)
    d, e = attn.dim_q, attn.dim_kv
    for pad in (0, 16, 3):
        wide = torch.zeros((3, d + 2 * e + 2 * pad), dtype=torch_dtype(dtype), device="cuda")
        views = wide[:, pad:pad + d], wide[:, pad + d:pad + d + e], wide[:, 2 * pad + d + e:]
        for t, x in zip(views, (q, k, v)):
            t.copy_(x)
        assert torch.equal(want, attn.step(cache, *views, lengths))
    for shift in (1, 4):                              # caches that begin inside another tensor
        for name in ("k", "v"):
            old = getattr(cache, name)
            flat = torch.zeros(old.numel() + shift, dtype=old.dtype, device="cuda")
            flat[shift:] = old.flatten()
            setattr(cache, name, flat[shift:].view(old.shape))
        assert torch.equal(want, attn.step(cache, q, k, v, lengths))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shared", [0, 45])
def test_a_prompt_and_its_tokens(dtype, shared):
    """Causal attention over whole sequences in one call, and the same as a prompt's first
    rows, the next rows after them, and then tokens on a cache."""
    irreps, heads, kv_heads, lens = "32x0e+16x1o", 4, 2, [50, 9, 33]
    first, then, tokens = [30, 2, 20], [15, 0, 8], 5
    attn = layers.CrossAttention(irreps, heads, kv_heads=kv_heads, dtype=dtype)
    rng = np.random.default_rng(9)
    ptr = ptr_of(lens)
    q = dev(rng.standard_normal((sum(lens), attn.dim_q)), dtype)
    k, v = (dev(rng.standard_normal((shared + sum(lens), attn.dim_kv)), dtype) for _ in range(2))
    whole = layers.Samples(ptr)
    want = attn.forward(attn.batch(whole, whole, causal=True, shared=shared), q, k, v)

    def rows(counts, skip):
        return torch.cat([torch.arange(ptr[s] + skip[s], ptr[s] + skip[s] + n, device="cuda") for s, n in enumerate(counts)])

    common = torch.arange(shared, device="cuda")
    got = torch.zeros_like(want)
    done = [0, 0, 0]
    for part in (first, then):
        held = [a + b for a, b in zip(done, part)]
        qi, ki = rows(part, done), torch.cat([common, shared + rows(held, [0, 0, 0])])
        b = attn.batch(layers.Samples(ptr_of(part)), layers.Samples(ptr_of(held)), causal=True, shared=shared)
        got[qi] = attn.forward(b, q[qi], k[ki], v[ki])
        done = held
    cache = attn.cache(3, 64, shared=shared)
    if shared:
        cache.share(k[:shared], v[:shared])
    for s, n in enumerate(done):
        at = slice(shared + ptr[s], shared + ptr[s] + n)
        cache.k[s, :n], cache.v[s, :n] = k[at], v[at]
    lengths = torch.tensor(done, dtype=torch.int32, device="cuda")
    for _ in range(tokens):
        qi = torch.tensor(ptr[:-1], device="cuda") + lengths
        got[qi] = attn.step(cache, q[qi], k[shared + qi], v[shared + qi], lengths)
        lengths += 1
    torch.cuda.synchronize()
    reached = [a + tokens for a in done]
    ri = rows(reached, [0, 0, 0])
    assert rel_err(host(got[ri]), host(want[ri])) <= TOL[dtype]
    for s, n in enumerate(reached):
        at = slice(shared + ptr[s], shared + ptr[s] + n)
        assert torch.equal(cache.k[s, :n], k[at]) and torch.equal(cache.v[s, :n], v[at])


@pytest.mark.parametrize("shared", [0, 600])
def test_captured_steps_count_on(shared):
    case = ("128x0e+128x1o", 8, 2, [0, 30, 500], 520, shared)
    attn, cache, q, k, v, lengths, common = setup(case, "bf16")
    twin = attn.cache(3, 520, shared=shared)
    twin.k.copy_(cache.k)
    twin.v.copy_(cache.v)
    twin._context = cache._context
    counts = lengths.clone()
    attn.step(twin, q, k, v, counts.clone())          # (writes the rows that the first replay writes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.step(cache, q, k, v, lengths)
        lengths.add_(1)
    for seed in range(24):                            # the third slot is full from the 21st on
        for t in (q, k, v):
            t.copy_(dev(np.random.default_rng(seed).standard_normal(t.shape), "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        want = attn.step(twin, q, k, v, counts)
        counts += 1
        assert torch.equal(got, want)
        assert torch.equal(cache.k, twin.k) and torch.equal(cache.v, twin.v)
    assert torch.all(got[2] == 0)


def test_caches_of_more_elements_than_32_bits_count():
    irreps, heads, lens = "128x0e+128x1o+128x2e+128x3o", 16, [5, 300, 20]
    case = (irreps, heads, heads, lens, 320, 0)
    attn, cache, q, k, v, lengths, common = setup(case, "bf16")
    big = attn.cache(3, 400000)                        # 2.5e9 elements each
    for a, b in ((cache.k, big.k), (cache.v, big.v)):
        b[:, :320] = a
    want, got = attn.step(cache, q, k, v, lengths), attn.step(big, q, k, v, lengths)
    torch.cuda.synchronize()
    assert rel_err(host(got), host(want)) <= TOL["bf16"]
    for s, n in enumerate(lens):
        assert torch.equal(big.k[s, :n + 2], cache.k[s, :n + 2]) and torch.equal(big.v[s, n], v[s])
    far = torch.tensor([-1, 0, 399999], dtype=torch.int32, device="cuda")
    attn.step(big, q, k, v, far)                       # the last place of all
    torch.cuda.synchronize()
    assert torch.equal(big.k[2, 399999], k[2]) and torch.equal(big.v[1, 0], v[1])


def test_two_streams_with_a_cache_each():
    case = ("32x0e+16x1o", 4, 2, [0, 5, 70], 90, 33)
    states = [setup(case, "bf16", seed) for seed in range(2)]
    want = [s[0].step(*s[1:6]) for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    got = []
    for st, s in zip(streams, states):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([s[0].step(*s[1:6]) for _ in range(5)])
    torch.cuda.synchronize()
    assert all(torch.equal(w, x) for w, g in zip(want, got) for x in g)


def test_refusals():
    attn = layers.CrossAttention("32x0e", 4, dtype="bf16")
    for bad in ((-1, 4, 0), (2, 0, 0), (2, -5, 0), (2, 4, -1)):
        with pytest.raises(cgtp.CgtpError) as e:
            attn.cache(bad[0], bad[1], shared=bad[2])
        assert e.value.status == 1
    for bad in ((2, 1 << 31, 0), (1, (1 << 30) + 1, 0), (1 << 31, 4, 0), (2, 4, 1 << 31), (1 << 20, 1 << 20, 0), (1 << 29, 1, 0)):
        with pytest.raises(cgtp.CgtpError) as e:
            attn.cache(bad[0], bad[1], shared=bad[2])
        assert e.value.status == 3
    cache = attn.cache(2, 8, shared=3)
    row = torch.zeros((2, 32), dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        attn.step(cache, row, row, row, n)            # nothing shared yet
    cache.share(torch.zeros((3, 32), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 32), dtype=torch.bfloat16, device="cuda"))
    attn.step(cache, row, row, row, n)
    for args in ((row.float(), row, row, n), (row[:1], row, row, n), (row, row, row[:, :16], n), (row, row, row, n.long()),
                 (row, row, row, n.cpu()), (row, None, row, n)):
        with pytest.raises(ValueError):
            attn.step(cache, *args)
    with pytest.raises(ValueError):
        layers.CrossAttention("32x0e", 4, dtype="bf16").step(cache, row, row, row, n)
    with pytest.raises(cgtp.CgtpError):
        attn.step(cache, row, row, row, n, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cgtp.CgtpError):
        attn.step(cache, row, row, row, n, scale=float("inf"))
    with pytest.raises(ValueError):
        cache.share(row, row)
    empty = attn.cache(0, 8)
    none = row[:0]
    assert attn.step(empty, none, none, none, n[:0]).shape == (0, 32)
