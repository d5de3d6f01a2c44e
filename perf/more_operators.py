"""Cases that time attention along sequences of irreps rows: causal attention
over whole prompts, attention of a batch that shares a long prefix, and a single
token's step on a growing cache.

Rows are irreps rows as everywhere in this package: blocks [2l+1][mul]
concatenated, channel index fastest. ``own`` false computes the operators from
elementary torch operations in fp32 (rounded once at the end); ``own`` true
calls clebsch_gordan_tensor_amd.layers.
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}

L2_32 = "32x0e+32x1o+32x2e"
L1_128 = "128x0e+128x1o"
L2_128 = "128x0e+128x1o+128x2e"
L3_128 = "128x0e+128x1o+128x2e+128x3o"
ODD = "35x0e+21x1o+7x2e"


# ------------------------------------------------------------------- cases
#
# op "batch": queries of lo .. hi rows a sample; their context is `shared` rows that
# every sample sees, then own rows: the queries' own after past_lo .. past_hi
# earlier ones (causal), or ctx_lo .. ctx_hi rows that all queries see.
# op "step": one new token a slot after lo .. hi cached ones, caches of `capacity`;
# every idle-th slot is not in use (0: all are).

def _causal(name, irreps, heads, kv_heads, dtype, kind, samples, lo, hi, past=(0, 0), shared=0):
    return dict(name=name, op="batch", irreps=irreps, heads=heads, kv_heads=kv_heads, dtype=dtype, kind=kind,
                causal=True, samples=samples, lo=lo, hi=hi, k_lo=past[0], k_hi=past[1], shared=shared, lens=1)


def _shared(name, irreps, heads, kv_heads, dtype, kind, samples, lo, hi, ctx, shared):
    return dict(name=name, op="batch", irreps=irreps, heads=heads, kv_heads=kv_heads, dtype=dtype, kind=kind,
                causal=False, samples=samples, lo=lo, hi=hi, k_lo=ctx[0], k_hi=ctx[1], shared=shared, lens=1)


def _step(name, irreps, heads, kv_heads, dtype, slots, lo, hi, capacity, shared=0, idle=0):
    return dict(name=name, op="step", irreps=irreps, heads=heads, kv_heads=kv_heads, dtype=dtype, kind="step",
                samples=slots, lo=lo, hi=hi, capacity=capacity, shared=shared, idle=idle, lens=1)


def listed():
    return [
        # a few short trajectories of one molecule's frames, inference: latency
        _causal("causal_small_f32", L2_32, 4, 4, "f32", "fwd", 8, 9, 40),
        # a training batch of trajectories of differing lengths, grouped heads
        _causal("causal_batch_bf16_train", L2_128, 8, 4, "bf16", "train", 24, 100, 1500),
        # one long trajectory, training in full precision
        _causal("causal_one_f32_train", L1_128, 4, 4, "f32", "train", 1, 3000, 3000),
        # whole long prompts before an answer, inference
        _causal("causal_long_bf16", L3_128, 16, 4, "bf16", "fwd", 4, 5000, 8191),
        # a prompt taken in chunks: the next rows of every sequence after what it holds
        _causal("causal_chunk_bf16", L3_128, 16, 4, "bf16", "fwd", 8, 500, 512, past=(1000, 6000)),
        # a few conformers, some atoms each, that read one surrounding and little of their own: latency
        _shared("shared_small_f32", L2_32, 4, 2, "f32", "fwd", 12, 1, 10, (0, 20), 50),
        # odd channel counts, seven heads on one context head, training with a common surrounding
        _shared("shared_odd_f32_train", ODD, 7, 1, "f32", "train", 9, 20, 300, (0, 100), 333),
        # a training batch of short trajectories after a common beginning
        _causal("shared_batch_bf16_train", L2_128, 8, 4, "bf16", "train", 32, 40, 200, shared=1500),
        # prompts that begin alike, inference
        _causal("shared_prompts_bf16", L3_128, 16, 4, "bf16", "fwd", 16, 100, 600, shared=6000),
        # a few short sequences, one token each: latency
        _step("step_small_f32", L2_32, 4, 4, "f32", 8, 5, 60, 64, idle=5),
        # serving: one token of each of many long sequences
        _step("step_batch_bf16", L3_128, 16, 4, "bf16", 64, 1000, 8000, 8192),
        # serving: answers to one long document, begun not long ago
        _step("step_shared_bf16", L3_128, 16, 4, "bf16", 64, 16, 500, 1024, shared=8000),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["causal", "causal", "shared", "shared", "step"])
    dtype = rng.choice(["f32", "bf16"])
    irreps, heads, kv_heads = rng.choice([(L2_32, 4, 4), (L2_32, 8, 2), (L1_128, 4, 4), (L1_128, 16, 4), (L2_128, 8, 8),
                                          (L2_128, 8, 4), (L3_128, 16, 16), (L3_128, 16, 4), (L3_128, 8, 8),
                                          (ODD, 7, 1), ("64x0e", 2, 2), ("256x0e", 2, 1)])
    common = dict(irreps=irreps, heads=heads, kv_heads=kv_heads, dtype=dtype, lens=rng.randrange(1 << 20))
    if kind == "step":
        slots = _spread(rng, 1, 64)
        row = _dim(_kv_irreps(common)) * _SIZE[dtype]
        hi = _spread(rng, 8, min(8000, 250000000 // (slots * row)))
        return dict(op="step", kind="step", samples=slots, lo=rng.choice([0, hi // 4, hi]), hi=hi,
                    capacity=hi + 1 + rng.randrange(200), shared=rng.choice([0, 0, _spread(rng, 20, 4000)]),
                    idle=rng.choice([0, 0, 3]), **common)
    pairs = _spread(rng, 1500, 15000000 if dtype == "bf16" else 3000000)
    samples = _spread(rng, 1, 32)
    shared = _spread(rng, 8, 4000) if kind == "shared" else 0
    causal = kind == "causal" or rng.random() < 0.5
    q = max(1, min(4000, int(math.sqrt(pairs / samples + shared * shared / 4.0) - shared / 2.0)))
    k = rng.choice([0, 0, q // 2, 3 * q]) if causal else _spread(rng, 1, q + 4)
    return dict(op="batch", kind=rng.choice(["fwd", "train"]), causal=causal, samples=samples, lo=max(0, q // 3),
                hi=q + q // 3, k_lo=k // 4, k_hi=k, shared=shared, **common)


# ----------------------------------------------------------------- shapes

def _blocks(irreps):
    """[(mul, 2l+1, element offset)] of an irreps string."""
    out, off = [], 0
    for term in irreps.split("+"):
        mul, lp = term.split("x")
        mul, l = int(mul), int(lp[:-1])
        out.append((mul, 2 * l + 1, off))
        off += mul * (2 * l + 1)
    return out


def _dim(irreps):
    return sum(mul * m for mul, m, _ in _blocks(irreps))


def _kv_irreps(case):
    """The context's irreps: as many channels a head, kv_heads heads."""
    r = case["heads"] // case["kv_heads"]
    return "+".join("%dx%s" % (int(t.split("x")[0]) // r, t.split("x")[1]) for t in case["irreps"].split("+"))


def _lengths(seed, n, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _batch_lengths(case):
    """(query rows, own context rows) of every sample."""
    nq = _lengths(case["lens"], case["samples"], case["lo"], case["hi"])
    nk = _lengths(case["lens"] + 1, case["samples"], case["k_lo"], case["k_hi"])
    return nq, [a + b for a, b in zip(nq, nk)] if case["causal"] else nk


def _step_lengths(case):
    """Cached tokens of every slot, -1 where it is not in use."""
    n = _lengths(case["lens"], case["samples"], case["lo"], case["hi"])
    return [-1 if case["idle"] and i % case["idle"] == case["idle"] - 1 else a for i, a in enumerate(n)]


def _ptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def work(case):
    es, H = _SIZE[case["dtype"]], case["heads"]
    dq, dk = _dim(case["irreps"]), _dim(_kv_irreps(case))
    d = dq // H
    if case["op"] == "step":
        used = [n for n in _step_lengths(case) if n >= 0]
        rows = sum(used) + (case["shared"] if used else 0)
        pairs = sum(n + 1 + case["shared"] for n in used)
        # q and out; cached and shared rows; the new rows read, and written to the cache
        return {"bytes": (2 * len(used) * dq + 2 * rows * dk + 4 * len(used) * dk) * es, "flops": 4 * d * H * pairs}
    nq, nk = _batch_lengths(case)
    if case["causal"]:
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(nq, nk))
    else:
        pairs = sum(a * b for a, b in zip(nq, nk))
    pairs = (pairs + case["shared"] * sum(nq)) * H
    q, k = sum(nq) * dq * es, (case["shared"] + sum(nk)) * dk * es
    if case["kind"] == "fwd":
        return {"bytes": 2 * q + 2 * k, "flops": 4 * d * pairs}
    # forward: q, k, v, out; backward: q, k, v, out, grad_out, and three gradients
    return {"bytes": (2 + 4) * q + (2 + 4) * k, "flops": 14 * d * pairs}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    dq, dk, P, S = _dim(case["irreps"]), _dim(_kv_irreps(case)), case["shared"], case["samples"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    st = dict(case=case)
    if case["op"] == "step":
        lens = _step_lengths(case)
        st["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"], st["k"], st["v"] = normal(S, dq), normal(S, dk), normal(S, dk)
        st["shared"] = (normal(P, dk), normal(P, dk)) if P else None
        keys, values = normal(S, case["capacity"], dk), normal(S, case["capacity"], dk)
        if own:
            from clebsch_gordan_tensor_amd import layers
            st["attn"] = layers.CrossAttention(case["irreps"], case["heads"], kv_heads=case["kv_heads"],
                                               dtype=case["dtype"])
            st["cache"] = st["attn"].cache(S, case["capacity"], shared=P)
            st["cache"].k.copy_(keys)
            st["cache"].v.copy_(values)
            if P:
                # the shared rows are encoded once and read by every token of every answer
                st["cache"].share(*st["shared"])
        else:
            st["keys"], st["values"] = keys, values
            st["slot"] = torch.arange(S, device="cuda")
            st["place"] = torch.arange(case["capacity"], device="cuda")
        return st
    nq, nk = _batch_lengths(case)
    st["q"] = normal(sum(nq), dq)
    st["k"], st["v"] = normal(P + sum(nk), dk), normal(P + sum(nk), dk)
    if case["kind"] == "train":
        st["grad"] = normal(sum(nq), dq)
    if own:
        from clebsch_gordan_tensor_amd import layers
        st["attn"] = layers.CrossAttention(case["irreps"], case["heads"], kv_heads=case["kv_heads"],
                                           dtype=case["dtype"])
        st["batch"] = st["attn"].batch(layers.Samples(_ptr(nq)), layers.Samples(_ptr(nk)), causal=case["causal"],
                                       shared=P)
    else:
        st["qpad"], st["kpad"] = _padding(nq, 0), _padding(nk, P)
        st["seen"] = torch.from_numpy(_seen(case, nq, nk)).cuda()
    return st


def _padding(lens, first):
    """(row index [S, longest] with 0 in the free places, mask of the used ones);
    the samples' rows come after `first` common ones."""
    ptr = first + np.array(_ptr(lens))
    idx = ptr[:-1, None] + np.arange(max(max(lens), 1))[None]
    used = idx < ptr[1:, None]
    if first:
        every = np.broadcast_to(np.arange(first), (len(lens), first))
        idx, used = np.concatenate([every, idx], 1), np.concatenate([every >= 0, used], 1)
    return torch.from_numpy(np.where(used, idx, 0)).cuda(), torch.from_numpy(used).cuda()


def _seen(case, nq, nk):
    """Which of the shared and own keys a query sees: [S, longest q], as a count of the own ones."""
    n = np.array(nk)[:, None] + 0 * np.arange(max(max(nq), 1))[None]
    if case["causal"]:
        n = n - np.array(nq)[:, None] + np.arange(n.shape[1])[None] + 1
    return n


# ------------------------------------------------------------------- passes

def run(st):
    case = st["case"]
    if case["op"] == "step":
        return _own_step(st) if own else _plain_step(st, case)
    return _own_batch(st, case) if own else _plain_batch(st, case)


def _own_batch(st, case):
    a, b = st["attn"], st["batch"]
    if case["kind"] == "fwd":
        return a.forward(b, st["q"], st["k"], st["v"])
    out, lse = a.forward(b, st["q"], st["k"], st["v"], need_lse=True)
    dq, dk, dv = a.backward(b, st["q"], st["k"], st["v"], out, lse, st["grad"])
    return out, dq, dk, dv


def _own_step(st):
    cache = st["cache"]
    return st["attn"].step(cache, st["q"], st["k"], st["v"], st["lengths"]), cache.k, cache.v


def _to_heads(x, irreps, heads):
    """[rows, dim] -> [rows, heads, head dim] in fp32."""
    return torch.cat([x[:, o:o + mul * m].float().view(-1, m, heads, mul // heads).transpose(1, 2)
                      .reshape(-1, heads, m * (mul // heads)) for mul, m, o in _blocks(irreps)], 2)


def _from_heads(x, irreps, heads):
    out, at = [], 0
    for mul, m, _ in _blocks(irreps):
        n = m * (mul // heads)
        out.append(x[:, :, at:at + n].reshape(-1, heads, m, mul // heads).transpose(1, 2).reshape(-1, m * mul))
        at += n
    return torch.cat(out, 1)


def _softmax(s, live):
    """Softmax over the live places of the last dimension, 0 where there is none."""
    s = s.masked_fill(~live, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _plain_batch(st, case):
    dt = st["q"].dtype
    H, Hk, P = case["heads"], case["kv_heads"], case["shared"]
    kvi = _kv_irreps(case)
    (qi, qu), (ki, ku) = st["qpad"], st["kpad"]
    zero = torch.zeros((), device="cuda")

    def queries(x):
        return _to_heads(x, case["irreps"], H)[qi].transpose(1, 2)                  # [S, H, nq, d]

    def keys(x):
        t = torch.where(ku[:, :, None, None], _to_heads(x, kvi, Hk)[ki], zero)
        return t.transpose(1, 2).repeat_interleave(H // Hk, 1)                        # [S, H, P + nk, d]

    q, k, v = queries(st["q"]), keys(st["k"]), keys(st["v"])
    # a query's own keys come after the shared ones, which all see
    place = torch.arange(ki.shape[1], device="cuda") - P
    live = (ku[:, None, :] & (place[None, None] < st["seen"][:, :, None]) | (place < 0)[None, None])[:, None]
    scale = 1.0 / math.sqrt(q.shape[-1])
    p = _softmax(torch.matmul(q, k.transpose(2, 3)) * scale, live)
    out = torch.matmul(p, v)

    def rows(x):
        return _from_heads(x.transpose(1, 2)[qu], case["irreps"], H).to(dt)

    if case["kind"] != "train":
        return rows(out)
    g = torch.where(qu[:, None, :, None], queries(st["grad"]), zero)
    dv = torch.matmul(p.transpose(2, 3), g)
    ds = p * (torch.matmul(g, v.transpose(2, 3)) - (g * out).sum(3, keepdim=True)) * scale
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)

    def context(x):
        S, _, n, d = x.shape
        x = x.view(S, Hk, H // Hk, n, d).sum(2).transpose(1, 2)                      # [S, P + nk, Hk, d]
        x = torch.cat([x[:, :P].sum(0), x[:, P:][ku[:, P:]]])
        return _from_heads(x, kvi, Hk).to(dt)

    return rows(out), rows(dq), context(dk), context(dv)


def _plain_step(st, case):
    dt = st["q"].dtype
    H, Hk, S, C, P = case["heads"], case["kv_heads"], case["samples"], case["capacity"], case["shared"]
    kvi = _kv_irreps(case)
    lens, slot = st["lengths"].long(), st["slot"]
    used = lens >= 0
    at = (slot, lens.clamp(min=0))

    def cached(cache, new):
        cache[at] = torch.where(used[:, None], new, cache[at])
        return _to_heads(cache.view(S * C, -1), kvi, Hk).view(S, C, Hk, -1).transpose(1, 2)    # [S, Hk, C, d]

    k, v = cached(st["keys"], st["k"]), cached(st["values"], st["v"])
    live = st["place"][None] <= lens[:, None]
    if P:
        k, v = (torch.cat([_to_heads(s, kvi, Hk).transpose(0, 1)[None].expand(S, -1, -1, -1), c], 2)
                for s, c in zip(st["shared"], (k, v)))
        live = torch.cat([used[:, None].expand(-1, P), live], 1)
    live = live[:, None, :, None]
    v = torch.where(live, v, torch.zeros((), device="cuda"))
    q = _to_heads(st["q"], case["irreps"], H)
    q = q.view(S, Hk, H // Hk, -1)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(q.shape[-1]))
    out = torch.matmul(_softmax(s, live.transpose(2, 3)), v)
    return _from_heads(out.reshape(S, H, -1), case["irreps"], H).to(dt), st["keys"], st["values"]


# -------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    return (_exact_step if case["op"] == "step" else _exact_batch)(case, prepare(case, seed))


def _columns(irreps, heads, h):
    return torch.cat([torch.arange(mul // heads) + off + j * mul + h * (mul // heads)
                      for mul, m, off in _blocks(irreps) for j in range(m)]).cuda()


def _exact_batch(case, st):
    H, Hk, P = case["heads"], case["kv_heads"], case["shared"]
    nq, nk = _batch_lengths(case)
    qp, kp = _ptr(nq), _ptr(nk)
    train = case["kind"] == "train"
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    for h in range(H):
        qc, kc = _columns(case["irreps"], H, h), _columns(_kv_irreps(case), Hk, h * Hk // H)
        scale = qc.numel() ** -0.5
        for s in range(case["samples"]):
            rows = torch.arange(qp[s], qp[s + 1], device="cuda")
            cols = torch.cat([torch.arange(P, device="cuda"), torch.arange(kp[s], kp[s + 1], device="cuda") + P])
            if not rows.numel() or not cols.numel():
                continue
            q = st["q"][rows][:, qc].double()
            k, v = st["k"][cols][:, kc].double(), st["v"][cols][:, kc].double()
            w = (q @ k.T) * scale
            if case["causal"]:
                # the last query sees the last key, each earlier one a key less
                hidden = torch.ones(nq[s], nk[s], dtype=torch.bool, device="cuda").triu(nk[s] - nq[s] + 1)
                w[:, P:][hidden] = -math.inf
            p = torch.softmax(w, 1)
            o = p @ v
            out[rows[:, None], qc[None]] = o
            if train:
                g = st["grad"][rows][:, qc].double()
                ds = p * (g @ v.T - (g * o).sum(1, keepdim=True)) * scale
                dq[rows[:, None], qc[None]] = ds @ k
                dk[cols[:, None], kc[None]] += ds.T @ q
                dv[cols[:, None], kc[None]] += p.T @ g
    return (out, dq, dk, dv) if train else out


def _exact_step(case, st):
    H, Hk = case["heads"], case["kv_heads"]
    keys, values = (st["cache"].k, st["cache"].v) if own else (st["keys"], st["values"])
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, n in enumerate(_step_lengths(case)):
        if n < 0:
            continue
        keys[s, n], values[s, n] = st["k"][s], st["v"][s]
        k, v = keys[s, :n + 1].double(), values[s, :n + 1].double()
        if case["shared"]:
            k, v = torch.cat([st["shared"][0].double(), k]), torch.cat([st["shared"][1].double(), v])
        for h in range(H):
            qc, kc = _columns(case["irreps"], H, h), _columns(_kv_irreps(case), Hk, h * Hk // H)
            w = (k[:, kc] @ st["q"][s, qc].double()) * qc.numel() ** -0.5
            out[s, qc] = torch.softmax(w, 0) @ v[:, kc]
    return out, keys.double(), values.double()
