"""Plain implementations of the operators that build, share and cross-read a paged cache, from their
definitions, on numpy arrays (attention in 64 bits, by tests/layer_reference.py)."""
import numpy as np

from tests import layer_reference as ref


def places(table, prefix_table, prefix_of, prefix_len, page):
    """Slot (page * page_size + place) of every position of every sequence, [n_seqs][capacity]."""
    B, cols = table.shape
    j = np.arange(cols * page)
    out = table.astype(np.int64)[:, j // page] * page + j % page
    for b in range(B):
        g = int(prefix_of[b])
        if 0 <= g < len(prefix_len):
            held = prefix_table.shape[1] * page
            i = j[:min(max(int(prefix_len[g]), 0), held)]
            out[b, i] = prefix_table[g].astype(np.int64)[i // page] * page + i % page
    return out


def attention(q, k, v, at, kv_len, q_start, n_heads, scale, window, sinks, every_key=False):
    """tests/layer_reference's attention with position j of sequence b in slot at[b][j]. every_key:
    each row sees all keys of its sequence."""
    flat = [x.reshape(-1, 1, *x.shape[2:]) for x in (k, v)]
    kv_len = np.clip(kv_len, 0, at.shape[1])
    if not every_key:
        return ref.attention(q, *flat, at, kv_len, q_start, n_heads, scale, window, sinks)
    seq = np.repeat(np.arange(len(kv_len)), np.diff(q_start))
    return ref.attention(q, *flat, at[seq], kv_len[seq], np.arange(len(seq) + 1), n_heads, scale,
                         0, 0)


def batch_tables(kv_len, n_new, spans, table, page, ring, state, T):
    """(q_start, slots, seqs, positions, kv_len, spans, state), table and ring changed in place."""
    B, cols = table.shape
    R = len(ring)
    head, count, _ = (int(x) for x in state)
    lens, spans = kv_len.copy(), spans.copy()
    q_start, rows = [0], []
    given, back, missing = 0, 0, 0
    was = ring.copy()
    for b in range(B):
        begin, end = (int(x) for x in spans[b])
        m, n = int(n_new[b]), int(kv_len[b])
        if m < 0:
            for col in range(begin, end):
                if count + back < R:
                    ring[(head + count + back) % R] = table[b, col]
                    back += 1
            lens[b] = 0
            spans[b] = 0
            q_start.append(q_start[-1])
            continue
        for col in range(end, min(-(-(n + m) // page), cols)):
            if given < count:
                table[b, col] = was[(head + given) % R]
                given += 1
                spans[b, 1] += 1
            else:
                table[b, col] = -1
                missing += 1
        lens[b] = n + m
        q_start.append(q_start[-1] + m)
        for pos in range(n, n + m):
            entry = int(table[b, pos // page]) if pos // page < cols else -1
            rows.append((entry * page + pos % page if entry >= 0 else -1, b, pos))
    rows = (rows + [(-1, -1, -1)] * T)[:T]
    slots, seqs, positions = np.array(rows, dtype=np.int64).reshape(-1, 3).T
    return (np.minimum(q_start, T), slots, seqs, positions, lens, spans,
            np.array([(head + given) % R, count - given + back, missing]))
