"""Plain 64-bit restatements of sampling, acceptance and the low-rank adapters, for the tests: loops and numpy, no
code of the library."""
import math

import numpy as np


def sample_row(logits, temp=1.0, top_k=0, top_p=1.0, min_p=0.0, u=0.5):
    """(token, logprob) of one row of fp64 logits; the parameters as the fp64 values of the stored fp32 ones."""
    l = np.where(np.isnan(logits), -np.inf, logits)
    ok = (temp == 0 or 2.0 ** -20 <= temp <= 2.0 ** 20) and top_p > 0 and min_p <= 1 and 0 <= u < 1
    live = np.flatnonzero(l > -np.inf)
    if not ok or not live.size:
        return -1, -math.inf
    order = live[np.argsort(-l[live], kind="stable")]
    top = l[order[0]]
    if temp == 0:
        return int(order[0]), 0.0
    x = np.array([0.0 if l[i] == top else (l[i] - top) / temp for i in order])
    w = np.exp(x)
    n = len(order)
    if top_k > 0:
        n = min(n, top_k)
    if top_p < 1:
        need, run, c = top_p * math.fsum(w[:n]), 0.0, 0
        while c < n and run < need:
            run += w[c]
            c += 1
        n = max(1, c)
    if min_p > 0:
        n = min(n, int(np.sum(w >= min_p)))
    kept = sorted(range(n), key=lambda r: order[r])
    total = math.fsum(w[:n])
    run = 0.0
    for r in kept:
        run += w[r]
        if run > u * total:
            return int(order[r]), float(x[r] - math.log(total))
    live_kept = [r for r in kept if w[r] > 0]
    return int(order[live_kept[-1]]), float(x[live_kept[-1]] - math.log(total))


def accept_row(draft, tokens, length, T):
    """(trim, next, emit) of one slot."""
    if not 1 <= length <= T:
        return -1, -1, [-1] * T
    n = 0
    while n + 1 < length and tokens[n] >= 0 and draft[n + 1] == tokens[n]:
        n += 1
    return T - 1 - n, tokens[n], list(tokens[:n + 1]) + [-1] * (T - n - 1)


def accept_tree_row(parent, draft, tokens, length, T):
    """(accept, next, emit, path) of one slot."""
    if not 0 <= length <= T:
        return -1, -1, [-1] * T, [-1] * T
    path, cur = [], 0 if length and parent[0] == -1 else -1
    while cur >= 0:
        path.append(cur)
        kids = [t for t in range(cur + 1, length) if parent[t] == cur and tokens[cur] >= 0 and draft[t] == tokens[cur]]
        cur = kids[0] if kids else -1
    last = path[-1] if path else -1
    pad = [-1] * (T - len(path))
    return last, tokens[last] if path else -1, [tokens[t] for t in path] + pad, path + pad


def lora(x, w, a, b, scale, ids, T):
    """(y, bound) for x [M][K], w [N][K], a [n][r][K], b [n][N][r] in fp64: the product with each slot's adapter,
    and how far a kernel with fp32 sums and one bf16 rounding may be off.  A sum of n fp32 products is off by at most
    n 2^-24 of the sum of their magnitudes (taken twice); h = A x enters B h with its own error and is carried as two
    bf16 numbers: the tail's half step is 2^-8 of at most 2^-8 of it."""
    y = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    K, r = x.shape[1], a.shape[1]
    err = K * 2.0 ** -23 * mag
    for s, i in enumerate(ids):
        if 0 <= i < a.shape[0]:
            rows = slice(s * T, (s + 1) * T)
            h = scale[i] * (x[rows] @ a[i].T)
            hm = abs(scale[i]) * (np.abs(x[rows]) @ np.abs(a[i]).T)
            y[rows] += h @ b[i].T
            err[rows] += ((K + 2 * r + 8) * 2.0 ** -23 * hm + 2.0 ** -16 * np.abs(h)) @ np.abs(b[i]).T
    return y, 2.0 ** -8 * (np.abs(y) + err) + err
