"""Float64 definitions of the vocabulary operators (numpy): logits of a 4-bit
W, log probabilities with entropy, rank and alternatives, their gradient, and
the embedding with its gradient.  Written from the formulas; used by the tests
only."""
import numpy as np


def unpack_w4(q):
    """[V, d / 2] bytes -> [V, d] integers 0..15 (low four bits first)."""
    q = np.asarray(q, np.uint8)
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.int64)
    out[:, 0::2] = q & 15
    out[:, 1::2] = q >> 4
    return out


def dequantise(q, scale, zero, group):
    """Weights scale * (q - zero) in float64; zero None means 8."""
    n = unpack_w4(q).astype(np.float64)
    z = 8.0 if zero is None else np.repeat(np.asarray(zero, np.float64), group, axis=1)
    return (n - z) * np.repeat(np.asarray(scale, np.float64), group, axis=1)


def clean_logits(l, n_valid_local=None, allow=None):
    """float64 logits with masked ids and NaN at -inf, +inf at the largest
    float32."""
    l = np.array(l, np.float64)
    V = l.shape[1]
    i = np.arange(V)
    ok = ~np.isnan(l)
    if n_valid_local is not None:
        ok &= (i < n_valid_local)[None, :]
    if allow is not None:
        ok &= ((np.asarray(allow, np.uint32)[:, i >> 5] >> (i & 31).astype(np.uint32)) & 1).astype(bool)
    l = np.minimum(l, float(np.finfo(np.float32).max))
    return np.where(ok, l, -np.inf)


def row_temps(temp, B, no_noise=False):
    if temp is None or no_noise:
        return np.ones(B)
    t = np.asarray(temp, np.float64)
    return np.where(t > 0, t, 1.0)


def logprobs(l, T, token, n_top, v_offset=0):
    """dict of logprob, rank, lse, entropy, top_idx, top_logprob of clean
    logits l [B, V]; x is the tempered row, absx and x2 the means of |x - m|
    and its square (for error bounds)."""
    B, V = l.shape
    r = dict(logprob=np.full(B, -np.inf), rank=np.zeros(B, np.int64), lse=np.full(B, -np.inf),
             entropy=np.zeros(B), top_idx=np.full((B, n_top), -1), absx=np.zeros(B), x2=np.zeros(B),
             top_logprob=np.full((B, n_top), -np.inf), m=np.zeros(B))
    for b in range(B):
        ids = np.nonzero(l[b] > -np.inf)[0]
        if ids.size == 0:
            continue
        m = l[b, ids].max()
        x = (l[b, ids] - m) / T[b]
        e = np.exp(x)
        S = e.sum()
        p = e / S
        xe = np.where(p > 0, x, 0.0)
        r["m"][b] = m / T[b]
        r["lse"][b] = m / T[b] + np.log(S)
        r["entropy"][b] = np.log(S) - (p * xe).sum()
        r["absx"][b], r["x2"][b] = (p * -xe).sum(), (p * xe * xe).sum()
        order = np.lexsort((ids, -l[b, ids]))[:n_top]
        r["top_idx"][b, :order.size] = ids[order] + v_offset
        r["top_logprob"][b, :order.size] = x[order] - np.log(S)
        t = -1 if token is None else int(token[b]) - v_offset
        if token is not None and token[b] >= 0 and 0 <= t < V and l[b, t] > -np.inf:
            r["logprob"][b] = (l[b, t] - m) / T[b] - np.log(S)
            r["rank"][b] = 1 + np.count_nonzero(l[b] > l[b, t]) + np.count_nonzero(l[b, :t] == l[b, t])
    return r


def logprobs_grad(l, T, token, top_idx, lse, entropy, g_logprob, g_lse, g_entropy, g_top, v_offset=0):
    """Gradient with respect to the logits, from the saved lse and entropy;
    and the magnitude that an error bound scales with."""
    B, V = l.shape
    out, mag = np.zeros((B, V)), np.zeros((B, V))
    for b in range(B):
        ok = l[b] > -np.inf
        if not np.isfinite(lse[b]):
            continue
        x = np.where(ok, l[b], 0.0) / T[b]
        lp = np.where(ok, x - lse[b], -np.inf)
        p = np.exp(lp)
        lpf = np.where(p > 0, lp, 0.0)
        c = 0.0 if g_lse is None else g_lse[b]
        ca = abs(c)
        gh = 0.0 if g_entropy is None else g_entropy[b]
        H = 0.0 if g_entropy is None else entropy[b]
        add = np.zeros(V)
        if g_logprob is not None and token[b] >= 0:
            c -= g_logprob[b]
            ca += abs(g_logprob[b])
            if 0 <= token[b] - v_offset < V:
                add[token[b] - v_offset] += g_logprob[b]
        if g_top is not None:
            for j in range(top_idx.shape[1]):
                if top_idx[b, j] >= 0:
                    c -= g_top[b, j]
                    ca += abs(g_top[b, j])
                    if 0 <= top_idx[b, j] - v_offset < V:
                        add[top_idx[b, j] - v_offset] += g_top[b, j]
        out[b] = np.where(ok, (p * (c - gh * (lpf + H)) + add) / T[b], 0.0)
        err = abs(lse[b]) + np.abs(x) + np.abs(lpf) + 16
        mag[b] = np.where(ok, (p * (ca + abs(gh) * (np.abs(lpf) + abs(H))) * err + 70 * np.abs(add)) / T[b], 0.0)
    return out, mag


def embed(ids, W, scale, v_offset=0):
    out = np.zeros((len(ids), W.shape[1]))
    for n, i in enumerate(np.asarray(ids, np.int64) - v_offset):
        if 0 <= i < W.shape[0]:
            out[n] = scale * W[i].astype(np.float64)
    return out


def embed_grad(ids, g, scale, V, v_offset=0):
    """Sums and the sums of absolute values (for error bounds)."""
    out, mag = np.zeros((V, g.shape[1])), np.zeros((V, g.shape[1]))
    for n, i in enumerate(np.asarray(ids, np.int64) - v_offset):
        if 0 <= i < V:
            out[i] += scale * g[n]
            mag[i] += abs(scale) * np.abs(g[n])
    return out, mag
