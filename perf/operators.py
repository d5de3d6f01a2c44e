"""Cases that time the layer operators on irreps rows: group norm with its
activation, cross attention to a context, dropout with a residual.

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

EPS = 1e-5
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}

L2_32 = "32x0e+32x1o+32x2e"
L1_128 = "128x0e+128x1o"
L2_128 = "128x0e+128x1o+128x2e"
L3_128 = "128x0e+128x1o+128x2e+128x3o"


# ------------------------------------------------------------------- cases

def _norm(name, irreps, groups, act, dtype, kind, samples, lo, hi):
    return dict(name=name, op="norm", irreps=irreps, groups=groups, act=act, dtype=dtype, kind=kind, samples=samples,
                lo=lo, hi=hi, lens=1)


def _drop(name, irreps, dtype, kind, rows, p, residual):
    return dict(name=name, op="dropout", irreps=irreps, dtype=dtype, kind=kind, rows=rows, p=p, residual=residual)


def _attn(name, irreps, heads, kv_heads, dtype, kind, samples, q_lo, q_hi, k_lo, k_hi, masked):
    return dict(name=name, op="attention", irreps=irreps, heads=heads, kv_heads=kv_heads, dtype=dtype, kind=kind,
                samples=samples, q_lo=q_lo, q_hi=q_hi, k_lo=k_lo, k_hi=k_hi, masked=masked, lens=1)


def listed():
    return [
        # inference on a handful of small molecules: latency
        _norm("norm_molecules_f32", L2_32, 4, "silu", "f32", "fwd", 8, 9, 21),
        # a training batch of molecules of differing sizes
        _norm("norm_batch_bf16_train", L2_128, 8, "silu", "bf16", "train", 96, 20, 220),
        # one large box (8000 waters) normalised as a whole, training in full precision
        _norm("norm_box_f32_train", L2_128, 8, "gelu", "f32", "train", 1, 24000, 24000),
        # many boxes of some thousand atoms at the widest rows, inference
        _norm("norm_boxes_bf16", L3_128, 4, "silu", "bf16", "fwd", 32, 1000, 6000),
        # odd channel counts, a small model on a single system of 1000 waters, training
        dict(_norm("norm_odd_f32_train", "35x0e+21x1o+7x2e", 7, "silu", "f32", "train", 3, 700, 3000)),
        # dropout of a small batch in the forward pass: latency
        _drop("dropout_small_f32", L2_32, "f32", "fwd", 168, 0.1, True),
        # a training step over the node rows of a large box, residual added
        _drop("dropout_large_bf16_train", L3_128, "bf16", "train", 1 << 18, 0.15, True),
        # one small system: a few atoms attend to a short context
        _attn("attn_small_f32", L2_32, 4, 4, "f32", "fwd", 8, 9, 21, 0, 60, 0.0),
        # ragged training batch, padded contexts (masked keys), grouped heads
        _attn("attn_batch_bf16_train", L2_128, 8, 4, "bf16", "train", 24, 100, 900, 50, 2000, 0.1),
        # the atoms of a 1000-water box attend to a context of some hundred states, full precision
        _attn("attn_box_f32_train", L1_128, 4, 4, "f32", "train", 1, 3000, 3000, 611, 611, 0.0),
        # long contexts, many queries, inference
        _attn("attn_long_bf16", L3_128, 16, 16, "bf16", "fwd", 4, 4096, 4096, 8191, 8191, 0.0),
        # serving: one new query a sample against contexts laid out once
        _attn("attn_token_bf16", L3_128, 16, 4, "bf16", "token", 64, 1, 1, 1000, 8000, 0.0),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "dropout", "attention"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "norm":
        irreps, groups = rng.choice([(L2_32, 4), (L2_32, 1), (L1_128, 8), (L2_128, 8), (L2_128, 16), (L3_128, 4),
                                     ("35x0e+21x1o+7x2e", 7), ("64x0e+24x0o+8x1e", 2)])
        total = _spread(rng, 40, 60000)
        samples = _spread(rng, 1, max(1, min(400, total // 8)))
        mean = max(1, total // samples)
        return dict(op=op, irreps=irreps, groups=groups, act=rng.choice(["silu", "gelu", "none"]), dtype=dtype,
                    kind=rng.choice(["fwd", "train"]), samples=samples, lo=max(0, mean // 3), hi=mean + mean // 2,
                    lens=rng.randrange(1 << 20))
    if op == "dropout":
        irreps = rng.choice([L2_32, L1_128, L2_128, L3_128, "35x0e+21x1o+7x2e", "256x0e"])
        return dict(op=op, irreps=irreps, dtype=dtype, kind=rng.choice(["fwd", "train"]),
                    rows=_spread(rng, 50, 100000), p=rng.choice([0.05, 0.1, 0.2, 0.5]), residual=rng.random() < 0.6)
    irreps, heads, kv_heads = rng.choice([(L2_32, 4, 4), (L2_32, 8, 2), (L1_128, 4, 4), (L1_128, 16, 4), (L2_128, 8, 8),
                                          (L2_128, 8, 4), (L3_128, 16, 16), (L3_128, 16, 4), (L3_128, 8, 8),
                                          ("35x0e+21x1o+7x2e", 7, 1), ("64x0e", 2, 2), ("256x0e", 2, 1)])
    kind = rng.choice(["fwd", "train", "token"])
    if kind == "token":
        samples = _spread(rng, 1, 64)
        q_lo = q_hi = 1
        k = _spread(rng, 20, 8000)
    else:
        pairs = _spread(rng, 2000, 6000000)
        samples = _spread(rng, 1, 32)
        q = _spread(rng, 4, max(4, min(4000, pairs // samples)))
        k = max(4, min(8000, pairs // (samples * q)))
        q_lo, q_hi = max(0, q // 3), q + q // 3
    return dict(op=op, irreps=irreps, heads=heads, kv_heads=kv_heads, dtype=dtype, kind=kind, samples=samples, q_lo=q_lo,
                q_hi=q_hi, k_lo=k // 4, k_hi=k, masked=rng.choice([0.0, 0.0, 0.15]), lens=rng.randrange(1 << 20))


# ----------------------------------------------------------------- shapes

def _blocks(irreps):
    """[(mul, 2l+1, is 0e, element offset, channel offset)] of an irreps string."""
    out, off, ch = [], 0, 0
    for term in irreps.split("+"):
        mul, lp = term.split("x")
        mul, l = int(mul), int(lp[:-1])
        out.append((mul, 2 * l + 1, lp == "0e", off, ch))
        off += mul * (2 * l + 1)
        ch += mul
    return out


def _dim(irreps):
    return sum(b[0] * b[1] for b in _blocks(irreps))


def _channels(irreps):
    return sum(b[0] for b in _blocks(irreps))


def _biases(irreps):
    return sum(b[0] for b in _blocks(irreps) if b[2])


def _kv_irreps(case):
    """The context's irreps: as many channels a head, kv_heads heads."""
    r = case["heads"] // case["kv_heads"]
    return "+".join("%dx%s" % (int(t.split("x")[0]) // r, t.split("x")[1]) for t in case["irreps"].split("+"))


def _lengths(seed, n, lo, hi):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _norm_lengths(case):
    return _lengths(case["lens"], case["samples"], case["lo"], case["hi"])


def _attn_lengths(case):
    return (_lengths(case["lens"], case["samples"], case["q_lo"], case["q_hi"]),
            _lengths(case["lens"] + 1, case["samples"], case["k_lo"], case["k_hi"]))


def _ptr(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def work(case):
    es = _SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = sum(_norm_lengths(case)) * _dim(case["irreps"])
        affine = (_channels(case["irreps"]) + _biases(case["irreps"])) * es
        if case["kind"] == "fwd":
            return {"bytes": 2 * n * es + affine, "flops": 10 * n}
        # forward: x, y; backward: x, grad_out, grad_x
        return {"bytes": 5 * n * es + 3 * affine, "flops": 30 * n}
    if case["op"] == "dropout":
        n = case["rows"] * _dim(case["irreps"])
        moved = (3 if case["residual"] else 2) * n
        if case["kind"] == "fwd":
            return {"bytes": moved * es, "flops": 2 * n}
        return {"bytes": (moved + 2 * n) * es, "flops": 3 * n}
    nq, nk = _attn_lengths(case)
    keep = 1.0 - case["masked"]
    pairs = sum(a * int(b * keep) for a, b in zip(nq, nk)) * case["heads"]
    d = _dim(case["irreps"]) // case["heads"]
    q, k = sum(nq) * _dim(case["irreps"]) * es, sum(nk) * _dim(_kv_irreps(case)) * es
    mask = sum(nk) if case["masked"] else 0
    if case["kind"] != "train":
        return {"bytes": 2 * q + 2 * k + mask, "flops": 4 * d * pairs}
    # forward: q, k, v, out; backward: q, k, v, out, grad_out, and three gradients
    return {"bytes": (2 + 4) * q + (2 + 4) * k + 2 * mask, "flops": 14 * d * pairs}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[case["dtype"]]
    irreps = case["irreps"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    st = dict(case=case)
    if case["op"] == "norm":
        lens = _norm_lengths(case)
        rows = sum(lens)
        # features of differing scale and, for the invariants, some offset
        x = torch.randn((rows, _dim(irreps)), generator=gen, device="cuda") * 1.5
        for mul, m, even, off, _ in _blocks(irreps):
            if even:
                x[:, off:off + mul] += 0.5
        st["x"] = x.to(dt)
        st["weight"] = (1.0 + 0.2 * torch.randn(_channels(irreps), generator=gen, device="cuda")).to(dt)
        st["bias"] = (0.2 * torch.randn(_biases(irreps), generator=gen, device="cuda")).to(dt)
        if case["kind"] == "train":
            st["grad"] = normal(rows, _dim(irreps))
        if own:
            from clebsch_gordan_tensor_amd import layers
            st["samples"] = layers.Samples(_ptr(lens))
            st["norm"] = layers.GroupNorm(irreps, case["groups"], activation=case["act"], eps=EPS, dtype=case["dtype"])
        else:
            st["pad"] = _padding(lens)
        return st
    if case["op"] == "dropout":
        st["x"] = normal(case["rows"], _dim(irreps))
        st["residual"] = normal(case["rows"], _dim(irreps)) if case["residual"] else None
        if case["kind"] == "train":
            st["grad"] = normal(case["rows"], _dim(irreps))
        r = random.Random(seed)
        st["seed"], st["offset"] = r.getrandbits(64), r.getrandbits(32)
        if own:
            from clebsch_gordan_tensor_amd import layers
            st["dropout"] = layers.Dropout(irreps, dtype=case["dtype"])
        return st
    nq, nk = _attn_lengths(case)
    kvi = _kv_irreps(case)
    st["q"] = normal(sum(nq), _dim(irreps))
    st["k"], st["v"] = normal(sum(nk), _dim(kvi)), normal(sum(nk), _dim(kvi))
    st["mask"] = None
    if case["masked"]:
        st["mask"] = torch.rand(sum(nk), generator=gen, device="cuda") >= case["masked"]
        # the last sample of a padded batch has an empty context
        if case["samples"] > 1:
            st["mask"][sum(nk) - nk[-1]:] = False
    if case["kind"] == "train":
        st["grad"] = normal(sum(nq), _dim(irreps))
    if own:
        from clebsch_gordan_tensor_amd import layers
        st["attn"] = layers.CrossAttention(irreps, case["heads"], kv_heads=case["kv_heads"], dtype=case["dtype"])
        st["batch"] = st["attn"].batch(layers.Samples(_ptr(nq)), layers.Samples(_ptr(nk)))
        if case["kind"] == "token":
            # the context is encoded once and read by every token of an answer
            st["context"] = st["attn"].pack(st["batch"], st["k"], st["v"], key_mask=st["mask"])
    else:
        st["qpad"], st["kpad"] = _padding(nq), _padding(nk)
    return st


def _padding(lens):
    """(row index [S, longest] with 0 in the free places, mask of the used ones)."""
    ptr = np.array(_ptr(lens))
    idx = ptr[:-1, None] + np.arange(max(max(lens), 1))[None]
    used = idx < ptr[1:, None]
    return torch.from_numpy(np.where(used, idx, 0)).cuda(), torch.from_numpy(used).cuda()


# ------------------------------------------------------------------- passes

def run(st):
    case = st["case"]
    return _OWN[case["op"]](st, case) if own else _PLAIN[case["op"]](st, case)


def _own_norm(st, case):
    y, stats = st["norm"].forward(st["samples"], st["x"], st["weight"], st["bias"])
    if case["kind"] == "fwd":
        return y
    gx, gw, gb = st["norm"].backward(st["samples"], st["x"], st["weight"], st["bias"], stats, st["grad"])
    return y, gx, gw, gb


def _own_dropout(st, case):
    y = st["dropout"].forward(st["x"], case["p"], st["seed"], st["offset"], residual=st["residual"])
    if case["kind"] == "fwd":
        return y
    return y, st["dropout"].backward(st["grad"], case["p"], st["seed"], st["offset"])


def _own_attention(st, case):
    a, b = st["attn"], st["batch"]
    if case["kind"] == "token":
        return a.forward_packed(b, st["q"], st["context"])
    if case["kind"] == "fwd":
        return a.forward(b, st["q"], st["k"], st["v"], key_mask=st["mask"])
    out, lse = a.forward(b, st["q"], st["k"], st["v"], key_mask=st["mask"], need_lse=True)
    dq, dk, dv = a.backward(b, st["q"], st["k"], st["v"], out, lse, st["grad"], key_mask=st["mask"])
    return out, dq, dk, dv


_OWN = {"norm": _own_norm, "dropout": _own_dropout, "attention": _own_attention}


def _act(z, act):
    """(activation, its derivative)"""
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2 * math.pi))
    return z, torch.ones_like(z)


def _plain_norm(st, case):
    dt = st["x"].dtype
    idx, used = st["pad"]
    S, n = idx.shape
    G = case["groups"]
    keep = used[:, :, None, None, None]
    count = used.sum(1).clamp(min=1).float()[:, None, None, None, None]
    x = st["x"].float()
    train = case["kind"] == "train"
    y = torch.empty_like(x)
    gx = torch.empty_like(x) if train else None
    gw, gb = [], []
    bias_at = 0
    for mul, m, even, off, ch in _blocks(case["irreps"]):
        c = mul // G
        cols = slice(off, off + mul * m)

        def padded(t):
            return torch.where(keep, t[:, cols][idx].view(S, n, m, G, c), torch.zeros((), device=t.device))

        total = count * (m * c)
        xb = padded(x)
        w = st["weight"][ch:ch + mul].float().view(G, c)
        if even:
            mean = xb.sum((1, 2, 4), keepdim=True) / total
            xb = torch.where(keep, xb - mean, torch.zeros((), device=x.device))
        rstd = torch.rsqrt((xb * xb).sum((1, 2, 4), keepdim=True) / total + EPS)
        xh = xb * rstd
        z = xh * w
        if even:
            z = z + st["bias"][bias_at:bias_at + mul].float().view(G, c)
            bias_at += mul
        a, da = _act(z, case["act"] if even else "none")
        y[:, cols] = a.reshape(S, n, m * mul)[used]
        if train:
            gz = padded(st["grad"].float()) * da
            ga, gc = (gz * xh).sum((1, 2)), gz.sum((1, 2))
            gw.append(ga.sum(0).reshape(-1))
            t = gz * w - xh * ((ga * w).sum(2)[:, None, None, :, None] / total)
            if even:
                gb.append(gc.sum(0).reshape(-1))
                t = t - (gc * w).sum(2)[:, None, None, :, None] / total
            gx[:, cols] = (t * rstd).reshape(S, n, m * mul)[used]
    if not train:
        return y.to(dt)
    none = torch.empty(0, device=x.device)
    return y.to(dt), gx.to(dt), torch.cat(gw).to(dt), torch.cat(gb + [none]).to(dt)


def _keep16(irreps, rows, seed, offset):
    """16-bit draws [rows, padded channels]: Philox 4x32 of 10 rounds, key = the
    seed, counter = (chunk of 8 channels, row low, row high, offset)."""
    m32 = 0xFFFFFFFF
    chunks = sum((b[0] + 7) // 8 for b in _blocks(irreps))
    c0 = torch.arange(chunks, device="cuda", dtype=torch.int64)[None, :].expand(rows, chunks)
    c1 = torch.arange(rows, device="cuda", dtype=torch.int64)[:, None].expand(rows, chunks)
    c2, c3 = torch.zeros_like(c0), torch.full_like(c0, offset)
    k0, k1 = seed & m32, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32, ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    words = torch.stack((c0, c1, c2, c3), 2)
    return torch.stack((words & 0xFFFF, words >> 16), 3).reshape(rows, chunks * 8)


def _plain_dropout(st, case):
    dt = st["x"].dtype
    t = int(math.floor(case["p"] * 65536 + 0.5))
    bits = _keep16(case["irreps"], case["rows"], st["seed"], st["offset"]) >= t
    scale = 65536.0 / (65536 - t)
    out, at = [], 0
    for mul, m, _, _, _ in _blocks(case["irreps"]):
        out.append(bits[:, None, at:at + mul].expand(-1, m, -1).reshape(case["rows"], m * mul))
        at += (mul + 7) // 8 * 8
    keep = torch.cat(out, 1)

    def apply(x):
        return torch.where(keep, x.float() * scale, torch.zeros((), device=x.device))

    y = apply(st["x"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    if case["kind"] == "fwd":
        return y.to(dt)
    return y.to(dt), apply(st["grad"]).to(dt)


def _to_heads(x, irreps, heads):
    """[rows, dim] -> [rows, heads, head dim] in fp32."""
    return torch.cat([x[:, o:o + mul * m].float().view(-1, m, heads, mul // heads).transpose(1, 2)
                      .reshape(-1, heads, m * (mul // heads)) for mul, m, _, o, _ in _blocks(irreps)], 2)


def _from_heads(x, irreps, heads):
    out, at = [], 0
    for mul, m, _, _, _ in _blocks(irreps):
        n = m * (mul // heads)
        out.append(x[:, :, at:at + n].reshape(-1, heads, m, mul // heads).transpose(1, 2).reshape(-1, m * mul))
        at += n
    return torch.cat(out, 1)


def _plain_attention(st, case):
    dt = st["q"].dtype
    H, Hk = case["heads"], case["kv_heads"]
    kvi = _kv_irreps(case)
    (qi, qu), (ki, ku) = st["qpad"], st["kpad"]
    live = ku if st["mask"] is None else ku & st["mask"][ki]
    zero = torch.zeros((), device="cuda")

    def queries(x):
        return _to_heads(x, case["irreps"], H)[qi].transpose(1, 2)                  # [S, H, nq, d]

    def keys(x):
        t = torch.where(live[:, :, None, None], _to_heads(x, kvi, Hk)[ki], zero)
        return t.transpose(1, 2).repeat_interleave(H // Hk, 1)                        # [S, H, nk, d]

    q, k, v = queries(st["q"]), keys(st["k"]), keys(st["v"])
    scale = 1.0 / math.sqrt(q.shape[-1])
    s = torch.matmul(q, k.transpose(2, 3)) * scale
    s = s.masked_fill(~live[:, None, None, :], -math.inf)
    top = s.amax(3, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, zero, top))
    del s
    total = p.sum(3, keepdim=True)
    p = p / torch.where(total == 0, zero + 1, total)
    out = torch.matmul(p, v)

    def rows(x):
        return _from_heads(x.transpose(1, 2)[qu], case["irreps"], H).to(dt)

    if case["kind"] != "train":
        return rows(out)
    g = torch.where(qu[:, None, :, None], queries(st["grad"]), zero)
    dv = torch.matmul(p.transpose(2, 3), g)
    ds = p * (torch.matmul(g, v.transpose(2, 3)) - (g * out).sum(3, keepdim=True)) * scale
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)

    def shared(x):
        S, _, n, d = x.shape
        return _from_heads(x.view(S, Hk, H // Hk, n, d).sum(2).transpose(1, 2)[ku], kvi, Hk).to(dt)

    return rows(out), rows(dq), shared(dk), shared(dv)


_PLAIN = {"norm": _plain_norm, "dropout": _plain_dropout, "attention": _plain_attention}


# -------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "dropout": _exact_dropout, "attention": _exact_attention}[case["op"]](st, case)


def _exact_norm(st, case):
    x, train = st["x"].double(), case["kind"] == "train"
    w, b = st["weight"].double(), st["bias"].double()
    y, gx = torch.zeros_like(x), torch.zeros_like(x)
    gw, gb = torch.zeros_like(w), torch.zeros_like(b)
    ptr = _ptr(_norm_lengths(case))
    for lo, hi in zip(ptr[:-1], ptr[1:]):
        if lo == hi:
            continue
        b_at = 0
        for mul, m, even, off, ch in _blocks(case["irreps"]):
            c = mul // case["groups"]
            shape = (hi - lo, m, case["groups"], c)
            xb = x[lo:hi, off:off + m * mul].reshape(shape)
            if even:
                xb = xb - xb.mean((0, 1, 3), keepdim=True)
            r = (xb.square().mean((0, 1, 3), keepdim=True) + EPS) ** -0.5
            xh, wb = xb * r, w[ch:ch + mul].view(case["groups"], c)
            z = xh * wb
            d = torch.ones_like(z)
            if even:
                z = z + b[b_at:b_at + mul].view(case["groups"], c)
                if case["act"] == "silu":
                    d = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
                elif case["act"] == "gelu":
                    d = 0.5 * torch.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
            out = z
            if even and case["act"] == "silu":
                out = z / (1 + torch.exp(-z))
            elif even and case["act"] == "gelu":
                out = z * 0.5 * torch.erfc(-z / 2 ** 0.5)
            y[lo:hi, off:off + m * mul] = out.reshape(hi - lo, m * mul)
            if train:
                gz = st["grad"][lo:hi, off:off + m * mul].double().reshape(shape) * d
                gw[ch:ch + mul] += (gz * xh).sum((0, 1)).view(-1)
                gh = gz * wb
                t = gh - xh * (gh * xh).mean((0, 1, 3), keepdim=True)
                if even:
                    gb[b_at:b_at + mul] += gz.sum((0, 1)).view(-1)
                    t = t - gh.mean((0, 1, 3), keepdim=True)
                gx[lo:hi, off:off + m * mul] = (t * r).reshape(hi - lo, m * mul)
            if even:
                b_at += mul
    return (y, gx, gw, gb) if train else y


def _exact_dropout(st, case):
    rows, blocks = case["rows"], _blocks(case["irreps"])
    chunks = sum(-(-b[0] // 8) for b in blocks)
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = [np.broadcast_to(np.arange(chunks, dtype=np.uint64)[None], (rows, chunks)),
           np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, chunks)),
           np.zeros((rows, chunks), np.uint64), np.full((rows, chunks), st["offset"], np.uint64)]
    key = [st["seed"] % (1 << 32), st["seed"] // (1 << 32)]
    for _ in range(10):
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> s32) ^ ctr[1] ^ np.uint64(key[0]), b & low, (a >> s32) ^ ctr[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    draws = np.ascontiguousarray(np.stack(ctr, 2).astype(np.uint32)).view(np.uint16).reshape(rows, chunks * 8)
    t = int(math.floor(case["p"] * 65536 + 0.5))
    kept = torch.from_numpy(draws >= t).cuda()
    factor = 1.0 / (1.0 - t / 65536)

    def masked(x):
        y, at = torch.zeros_like(x, dtype=torch.float64), 0
        for mul, m, _, off, _ in blocks:
            for k in range(m):
                cols = slice(off + k * mul, off + (k + 1) * mul)
                y[:, cols] = x[:, cols].double() * kept[:, at:at + mul] * factor
            at += -(-mul // 8) * 8
        return y

    y = masked(st["x"])
    if st["residual"] is not None:
        y += st["residual"].double()
    return (y, masked(st["grad"])) if case["kind"] == "train" else y


def _exact_attention(st, case):
    H, Hk = case["heads"], case["kv_heads"]
    nq, nk = _attn_lengths(case)
    qp, kp = _ptr(nq), _ptr(nk)
    train = case["kind"] == "train"
    blocks, kblocks = _blocks(case["irreps"]), _blocks(_kv_irreps(case))
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(out)
    dk = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)

    def columns(bl, heads, h):
        return torch.cat([torch.arange(mul // heads) + off + j * mul + h * (mul // heads)
                          for mul, m, _, off, _ in bl for j in range(m)]).cuda()

    for h in range(H):
        qc, kc = columns(blocks, H, h), columns(kblocks, Hk, h // (H // Hk))
        scale = qc.numel() ** -0.5
        for s in range(case["samples"]):
            rows = torch.arange(qp[s], qp[s + 1], device="cuda")
            cols = torch.arange(kp[s], kp[s + 1], device="cuda")
            if st["mask"] is not None:
                cols = cols[st["mask"][kp[s]:kp[s + 1]]]
            if not rows.numel() or not cols.numel():
                continue
            q = st["q"][rows][:, qc].double()
            k, v = st["k"][cols][:, kc].double(), st["v"][cols][:, kc].double()
            p = torch.softmax((q @ k.T) * scale, 1)
            o = p @ v
            out[rows[:, None], qc[None]] = o
            if train:
                g = st["grad"][rows][:, qc].double()
                ds = p * (g @ v.T - (g * o).sum(1, keepdim=True)) * scale
                dq[rows[:, None], qc[None]] = ds @ k
                dk[cols[:, None], kc[None]] += ds.T @ q
                dv[cols[:, None], kc[None]] += p.T @ g
    return (out, dq, dk, dv) if train else out
