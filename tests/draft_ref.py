"""Plain 64-bit definitions of what checks drafted tokens, on the CPU (numpy).
Nothing here calls the library."""
import numpy as np


def chains(parents):
    """For each token its chain: itself, its parent, and so on; and its depth.
    A parent that does not stand before its token is none."""
    out = []
    for i, p in enumerate(parents):
        out.append([i] + (out[p] if 0 <= p < i else []))
    return out, [len(c) - 1 for c in out]


def tree_arrays(parents_of, words):
    """seen (rows x words uint64) and depth of a batch's sequences; tokens from
    64 * words on see none of the new tokens, at depth 0."""
    seen, depth = [], []
    for parents in parents_of:
        most = 64 * words
        c, d = chains(parents[:most])
        for i in range(len(parents)):
            w = [0] * words
            for j in (c[i] if i < most else ()):
                w[j // 64] |= 1 << (j % 64)
            seen.append(w)
            depth.append(d[i] if i < most else 0)
    return np.array(seen, np.uint64).reshape(-1, words), np.array(depth, np.int32)


def attention_tree64(q, batch, parents_of, kv, vv, n_kv, scale, softcap=0.0, window=0, slopes=None, prefix=None):
    """As kv_ref.attention64, for a batch whose sequences' new tokens are trees."""
    N, n_q, D = q.shape
    out, T = np.zeros((N, n_q, D)), np.zeros((N, n_q, D))
    A = np.zeros((N, n_q, 1))
    G = n_q // n_kv
    trees = [chains(p) for p in parents_of]
    for row, s, index in batch.tokens():
        L, base = kv[s].shape[0], batch.len[s] - batch.new[s]
        chain, depth = trees[s]
        i = index - base
        j = np.arange(L)
        place = np.array([x if x < base else base + depth[x - base] for x in range(L)], np.int64)
        p = base + depth[i]
        seen = (j < base) | np.isin(j, [base + x for x in chain[i]])
        if window:
            seen = seen & (p - place < window)
        if prefix is not None:
            seen = seen | (j < prefix[s])
        if not seen.any():
            continue
        jj = j[seen]
        for h in range(n_q):
            k, v = kv[s][jj, h // G], vv[s][jj, h // G]
            x = q[row, h].astype(np.float64)
            t = scale * (k @ x)
            A[row, h] = abs(scale) * (np.abs(k) @ np.abs(x)).max()
            if softcap:
                t = softcap * np.tanh(t / softcap)
            if slopes is not None:
                t = t - np.float64(slopes[h]) * np.abs(p - place[jj])
            w = np.exp(t - t.max())
            w /= w.sum()
            out[row, h], T[row, h] = w @ v, w @ np.abs(v)
    return out, T, A


def logprobs64(logits, scale=1.0, softcap=0.0):
    """(log probabilities, entropy, order of the tokens) of fp32 or bf16-valued rows."""
    x = np.asarray(logits, np.float64)
    order = np.argsort(-x, axis=1, kind="stable")
    if softcap:
        x = np.where(np.isneginf(x), x, softcap * np.tanh(x / softcap))
    x = x * scale
    top = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        lp = np.where(np.isneginf(top), -np.inf, x - top - np.log(np.exp(x - np.where(np.isneginf(top), 0, top)).sum(1, keepdims=True)))
        h = -np.where(np.isneginf(lp), 0.0, np.exp(lp) * lp).sum(1)
    return lp, h, order
