"""Layers on irreps rows: group norm with activation, dropout, cross attention
(oracle; test infrastructure). fp64 NumPy from the definitions, loops over
samples, blocks, groups and heads."""

import math

import numpy as np

from .irreps import block_offsets, parse_irreps


def blocks(irreps):
    """[(mul, l, parity, element offset, channel offset, bias offset or None)]"""
    ir = parse_irreps(irreps)
    out, ch, bias = [], 0, 0
    for (mul, l, p), off in zip(ir, block_offsets(ir)):
        even = l == 0 and p > 0
        out.append((mul, l, p, off, ch, bias if even else None))
        ch += mul
        bias += mul if even else 0
    return out


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    if name == "silu":
        return z / (1.0 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    return z


def act_slope(z, name):
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def _norm_blocks(irreps, groups, ptr):
    for s in range(len(ptr) - 1):
        if ptr[s] == ptr[s + 1]:
            continue
        for mul, l, _, off, ch, bias in blocks(irreps):
            c = mul // groups
            for g in range(groups):
                # element columns [2l+1][c] and channels of the group
                cols = off + np.arange(2 * l + 1)[:, None] * mul + g * c + np.arange(c)[None]
                yield s, slice(ptr[s], ptr[s + 1]), cols, ch + g * c + np.arange(c), \
                    None if bias is None else bias + g * c + np.arange(c)


def _normalised(x, rows, cols, biased, eps):
    xb = x[rows][:, cols]                        # [n, 2l+1, c]
    mu = xb.mean() if biased else 0.0
    r = 1.0 / math.sqrt(((xb - mu) ** 2).mean() + eps)
    return (xb - mu) * r, mu, r


def norm_forward(irreps, groups, ptr, x, w, b, eps, name):
    y = np.zeros_like(x)
    for _, rows, cols, ch, bc in _norm_blocks(irreps, groups, ptr):
        xh, _, _ = _normalised(x, rows, cols, bc is not None, eps)
        z = xh * w[ch]
        if bc is not None:
            z = act(z + b[bc], name)
        y[rows, cols.reshape(-1)] = z.reshape(z.shape[0], -1)
    return y


def norm_backward(irreps, groups, ptr, x, w, b, eps, name, g):
    gx, gw, gb = np.zeros_like(x), np.zeros_like(w), np.zeros_like(b)
    for _, rows, cols, ch, bc in _norm_blocks(irreps, groups, ptr):
        xh, _, r = _normalised(x, rows, cols, bc is not None, eps)
        gz = g[rows][:, cols]
        if bc is not None:
            gz = gz * act_slope(xh * w[ch] + b[bc], name)
            gb[bc] += gz.sum((0, 1))
        gw[ch] += (gz * xh).sum((0, 1))
        gh = gz * w[ch]
        d = gh - xh * (gh * xh).mean()
        if bc is not None:
            d = d - gh.mean()
        gx[rows, cols.reshape(-1)] = (d * r).reshape(d.shape[0], -1)
    return gx, gw, gb


def philox(counter, key):
    """Philox 4x32 with 10 rounds of one counter (4 words) and key (2 words)."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def dropout_mask(irreps, rows, p, seed, offset):
    """keep [len(rows), dim] (bool) for row indices ``rows``, and the scale."""
    t = min(65535, int(math.floor(p * 65536 + 0.5)))
    out = []
    for r in rows:
        line, chunk = [], 0
        for mul, l, _, _, _, _ in blocks(irreps):
            ch = []
            for c in range(0, mul, 8):
                wd = philox((chunk, r & 0xFFFFFFFF, r >> 32, offset), (seed & 0xFFFFFFFF, seed >> 32))
                ch += [((wd[i // 2] >> (16 * (i % 2))) & 0xFFFF) >= t for i in range(min(8, mul - c))]
                chunk += 1
            line += ch * (2 * l + 1)
        out.append(line)
    return np.array(out, bool).reshape(len(out), -1), 65536.0 / (65536 - t)


def head_columns(irreps, heads, h):
    """Columns of head h: its channels of every block, all components."""
    return np.concatenate([off + m * mul + h * (mul // heads) + np.arange(mul // heads)
                           for mul, l, _, off, _, _ in blocks(irreps) for m in range(2 * l + 1)])


def kv_irreps(irreps, heads, kv_heads):
    return "+".join("%dx%d%s" % (mul * kv_heads // heads, l, "e" if p > 0 else "o")
                    for mul, l, p, _, _, _ in blocks(irreps))


def _attn_pairs(irreps, heads, kv_heads, qptr, kptr, mask):
    kvi = kv_irreps(irreps, heads, kv_heads)
    for s in range(len(qptr) - 1):
        rows = np.arange(qptr[s], qptr[s + 1])
        keys = np.arange(kptr[s], kptr[s + 1])
        if mask is not None:
            keys = keys[mask[keys] != 0]
        for h in range(heads):
            yield rows, keys, h, np.ix_(rows, head_columns(irreps, heads, h)), \
                np.ix_(keys, head_columns(kvi, kv_heads, h * kv_heads // heads))


def attn_forward(irreps, heads, kv_heads, qptr, kptr, q, k, v, mask, scale):
    """(out, lse)"""
    out = np.zeros_like(q)
    lse = np.full((q.shape[0], heads), -np.inf)
    for rows, keys, h, qi, ki in _attn_pairs(irreps, heads, kv_heads, qptr, kptr, mask):
        if not len(rows) or not len(keys):
            continue
        s = scale * (q[qi] @ k[ki].T)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        out[qi] = (e / e.sum(1, keepdims=True)) @ v[ki]
        lse[rows, h] = np.log(e.sum(1)) + top[:, 0]
    return out, lse


def attn_backward(irreps, heads, kv_heads, qptr, kptr, q, k, v, mask, scale, g):
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    out, lse = attn_forward(irreps, heads, kv_heads, qptr, kptr, q, k, v, mask, scale)
    for rows, keys, h, qi, ki in _attn_pairs(irreps, heads, kv_heads, qptr, kptr, mask):
        if not len(rows) or not len(keys):
            continue
        p = np.exp(scale * (q[qi] @ k[ki].T) - lse[rows, h][:, None])
        ds = p * (g[qi] @ v[ki].T - (g[qi] * out[qi]).sum(1, keepdims=True)) * scale
        dq[qi] += ds @ k[ki]
        dk[ki] += ds.T @ q[qi]
        dv[ki] += p.T @ g[qi]
    return dq, dk, dv


def _seq_pairs(irreps, heads, kv_heads, qptr, kptr, mask, causal, shared):
    """Per sample and head: rows, seen [rows, keys], head, indices into q and into k, v."""
    kvi = kv_irreps(irreps, heads, kv_heads)
    for s in range(len(qptr) - 1):
        rows = np.arange(qptr[s], qptr[s + 1])
        n, nq = kptr[s + 1] - kptr[s], len(rows)
        keys = np.concatenate([np.arange(shared), shared + kptr[s] + np.arange(n)]).astype(int)
        seen = np.ones((nq, len(keys)), bool)
        if causal:
            for i in range(nq):
                seen[i, shared + max(0, min(n, i + n - nq + 1)):] = False
        if mask is not None:
            seen &= mask[keys] != 0
        for h in range(heads):
            yield rows, seen, h, np.ix_(rows, head_columns(irreps, heads, h)), \
                np.ix_(keys, head_columns(kvi, kv_heads, h * kv_heads // heads))


def seq_forward(irreps, heads, kv_heads, qptr, kptr, q, k, v, mask, scale, causal=False, shared=0):
    """(out, lse) of queries that see the first `shared` rows of k and v and their own
    sample's after them, causally or whole."""
    out = np.zeros_like(q)
    lse = np.full((q.shape[0], heads), -np.inf)
    for rows, seen, h, qi, ki in _seq_pairs(irreps, heads, kv_heads, qptr, kptr, mask, causal, shared):
        s = scale * (q[qi] @ k[ki].T)
        for r, i in enumerate(rows):
            at = np.flatnonzero(seen[r])
            if not len(at):
                continue
            top = s[r, at].max()
            e = np.exp(s[r, at] - top)
            out[i, qi[1][0]] = e @ v[ki][at] / e.sum()
            lse[i, h] = np.log(e.sum()) + top
    return out, lse


def seq_backward(irreps, heads, kv_heads, qptr, kptr, q, k, v, mask, scale, g, causal=False, shared=0):
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    out, lse = seq_forward(irreps, heads, kv_heads, qptr, kptr, q, k, v, mask, scale, causal, shared)
    for rows, seen, h, qi, ki in _seq_pairs(irreps, heads, kv_heads, qptr, kptr, mask, causal, shared):
        top = np.where(np.isinf(lse[rows, h]), 0.0, lse[rows, h])
        p = np.where(seen, np.exp(np.where(seen, scale * (q[qi] @ k[ki].T), 0.0) - top[:, None]), 0.0)
        ds = p * (g[qi] @ v[ki].T - (g[qi] * out[qi]).sum(1, keepdims=True)) * scale
        dq[qi] += ds @ k[ki]
        dk[ki] += ds.T @ q[qi]
        dv[ki] += p.T @ g[qi]
    return dq, dk, dv


def cache_step(irreps, heads, kv_heads, q, k, v, k_cache, v_cache, lengths, scale, shared=None):
    """(out, lse, k_cache, v_cache): a token of every slot put at its length; `shared`:
    (keys, values, mask) of rows that all slots see first."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    out, lse = np.zeros_like(q), np.full((len(q), heads), -np.inf)
    for s, n in enumerate(lengths):
        if not 0 <= n < k_cache.shape[1]:
            continue
        k_cache[s, n], v_cache[s, n] = k[s], v[s]
        keys, values, mask = k_cache[s, :n + 1], v_cache[s, :n + 1], np.ones(n + 1)
        if shared is not None:
            keys, values = np.concatenate([shared[0], keys]), np.concatenate([shared[1], values])
            mask = np.concatenate([np.ones(len(shared[0])) if shared[2] is None else shared[2], mask])
        o, l = attn_forward(irreps, heads, kv_heads, [0, 1], [0, len(keys)], q[s:s + 1], keys, values, mask, scale)
        out[s], lse[s] = o[0], l[0]
    return out, lse, k_cache, v_cache
