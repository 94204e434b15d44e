"""Plain implementations in 64 bits of the operators between a decoder layer's linears, from their
definitions, on numpy arrays; and the error bounds their fp32 / bf16 results are held to.

The cache arrives as [n_pages][page_size][n_kv][D] and a page table, exactly as the library sees
it; nothing here shares code with the library."""
import numpy as np

F32 = 2.0 ** -24  # half an ulp of fp32 (24 significant bits), relative
BF16 = 2.0 ** -8  # half an ulp of bf16 (8 significant bits), relative


def rows_of(q_start, kv_len, capacity):
    """(row, sequence, position) of every token row."""
    out = []
    for b in range(len(kv_len)):
        n = min(max(int(kv_len[b]), 0), capacity)
        m = int(q_start[b + 1]) - int(q_start[b])
        out += [(int(q_start[b]) + i, b, n - m + i) for i in range(m)]
    return out


def visible(pos, window, sinks):
    if pos < 0:
        return np.zeros(0, dtype=np.int64)
    j = np.arange(pos + 1)
    if window > 0:
        j = j[(j > pos - window) | (j < sinks)]
    return j


def attention(q, k, v, table, kv_len, q_start, n_heads, scale, window, sinks):
    """y [T][n_heads][D], lse [T][n_heads], a = sum p |v| [T][n_heads][D] (what a relative error of
    the weights p can move y by), ds [T][n_heads] (a bound on the error of a score whose products
    are summed in fp32 in any order) and the number of visible keys."""
    n_pages, page, n_kv, D = k.shape
    T = q.shape[0]
    y = np.zeros((T, n_heads, D))
    a = np.zeros((T, n_heads, D))
    lse = np.full((T, n_heads), -np.inf)
    ds = np.zeros((T, n_heads))
    count = np.zeros((T, 1))
    G = n_heads // n_kv
    for t, b, pos in rows_of(q_start, kv_len, table.shape[1] * page):
        j = visible(pos, window, sinks)
        count[t] = len(j)
        if len(j) == 0:
            continue
        at = (table[b][j // page], j % page)
        for h in range(n_heads):
            kk, vv = k[at][:, h // G], v[at][:, h // G]
            qq = q[t].reshape(n_heads, D)[h]
            s = scale * (kk @ qq)
            e = np.exp(s - s.max())
            p = e / e.sum()
            y[t, h] = p @ vv
            a[t, h] = p @ np.abs(vv)
            lse[t, h] = s.max() + np.log(e.sum())
            ds[t, h] = (D + 4) * F32 * scale * (np.abs(kk) @ np.abs(qq)).max() \
                + 8 * F32 * np.abs(s).max()
    return y, lse, a, ds, count


def attention_bound(a, ds, count, weight_bits):
    """|y - y_ref| of an fp32 result: the scores' error moves a weight by at most 2 ds (its own and
    the sum's), the weights are held to `weight_bits`, the exponential to 2^-20, the sums run over
    `count` keys in fp32."""
    rel = 2.2 * ds + 2.0 ** -weight_bits + 2.0 ** -20 + 4 * count * F32
    return a * rel[..., None] + 1e-30


def rope(x, pos, inv_freq, layout, factor):
    """x [T][H][D] -> the rotated heads, and |a| + |b| of each value's pair."""
    R = 2 * len(inv_freq)
    t = pos[:, None, None].astype(np.float64) * inv_freq.astype(np.float64)
    c, s = factor * np.cos(t), factor * np.sin(t)
    if layout == 0:
        ia, ib = np.arange(R // 2), np.arange(R // 2) + R // 2
    else:
        ia, ib = np.arange(0, R, 2), np.arange(1, R, 2)
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def rms(u, w, eps, offset):
    return u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * (w + offset)


def residual_norm(x, r, w_pre, w_post, gate, alpha, eps, offset):
    """(y, r', |r| + |alpha g n|)."""
    if x is None:
        return rms(r, w_pre, eps, offset), r, np.abs(r)
    n = x if w_post is None else rms(x, w_post, eps, offset)
    add = alpha * n if gate is None else alpha * gate * n
    return rms(r + add, w_pre, eps, offset), r + add, np.abs(r) + np.abs(add)
