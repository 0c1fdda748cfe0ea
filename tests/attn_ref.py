"""The paged cache, the append and the attention as plain 64-bit loops over slots, and inputs to try them on."""
import math

import torch

import gated_deltanet_verify_gb300 as gdn

NAN = float("nan")


class Case:
    """One batch: sizes, the slots' pasts and real lengths, and whether it is a tree."""

    def __init__(self, T, H, Hk, D, page, past, length=None, dtype="bf16", tree=False, window=0, n_sink=0, scale=None,
                 gap=0, seed=0):
        self.B, self.T, self.H, self.Hk, self.D, self.page = len(past), T, H, Hk, D, page
        self.past, self.length = list(past), list(length) if length is not None else None
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.tree, self.window, self.n_sink = tree, window, n_sink
        self.scale = D ** -0.5 if scale is None else scale
        self.gap = gap                                     # elements between a page and the next, in page_stride
        self.g = torch.Generator().manual_seed(seed)
        self.half = torch.finfo(self.dtype).eps / 2

    def n(self, s):
        return self.T if self.length is None else self.length[s]

    def rand(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.g) * std).to(self.dtype)

    def pages(self, junk=(-1, 2 ** 31 - 1, -2 ** 31)):
        """A page table in a random order; junk in the entries behind a slot's last page."""
        need = [-(-(p + self.n(s)) // self.page) for s, p in enumerate(self.past)]
        self.max_pages, self.n_pages = max(max(need), 1) + 1, sum(need) + 2
        order = torch.randperm(self.n_pages, generator=self.g).tolist()
        self.table = torch.empty((self.B, self.max_pages), dtype=torch.int32)
        for s in range(self.B):
            for i in range(self.max_pages):
                self.table[s, i] = order.pop() if i < need[s] else junk[(s + i) % len(junk)]

    def where(self, s, p):
        return int(self.table[s, p // self.page]), p % self.page

    def pool(self, fill=NAN):
        """[n_pages][page_stride] with a page's rows [Hk][page][D] at its start."""
        flat = torch.full((self.n_pages, self.Hk * self.page * self.D + self.gap), fill, dtype=self.dtype)
        return flat

    def rows(self, flat):
        return flat[:, :self.Hk * self.page * self.D].view(self.n_pages, self.Hk, self.page, self.D)

    def parents(self):
        """Random trees in token order: node 0 a root, few other roots."""
        parent = torch.full((self.B, self.T), -1, dtype=torch.int32)
        for s in range(self.B):
            for t in range(1, self.T):
                low = max(-1 if t % 7 == 3 else 0, t - 6)
                parent[s, t] = int(torch.randint(low, t, (1,), generator=self.g))
        return parent

    def dims(self):
        return gdn.make_attn_dims(self.B, self.T, self.H, self.Hk, self.D, self.page, self.n_pages, self.max_pages,
                                  page_stride=self.Hk * self.page * self.D + self.gap,
                                  dtype=gdn.GDN_BF16 if self.dtype == torch.bfloat16 else gdn.GDN_F32)


def line(parent, t):
    """Node t and its ancestors."""
    out = []
    while t >= 0:
        out.append(t)
        t = int(parent[t])
    return out


def attend_ref(c, q, k, v, parent=None):
    """k, v: per slot [positions][Hk][D] (storage order).  Returns per slot (out, magnitude, reach): the output [n][H][D]
    in 64 bits, sum w |v| / sum w beside it, and the largest sum |q k| of a score (all for the tolerance)."""
    res = []
    G = c.H // c.Hk
    for s in range(c.B):
        n, past = c.n(s), c.past[s]
        if n == 0:
            res.append(None)
            continue
        N = past + n
        see = torch.zeros((n, N), dtype=torch.bool)
        position = list(range(past)) + [past + (len(line(parent[s], t)) - 1 if c.tree else t) for t in range(n)]
        where = torch.tensor(position)
        for t in range(n):
            see[t, :past] = True
            for u in (line(parent[s], t) if c.tree else range(t + 1)):
                see[t, past + u] = True
            if c.window:
                see[t] &= (position[past + t] - where < c.window) | (where < c.n_sink)
        qs, ks, vs = (x.double() for x in (q[s, :n], k[s], v[s]))
        ks, vs = ks.repeat_interleave(G, 1), vs.repeat_interleave(G, 1)
        x = torch.einsum("thd,nhd->htn", qs, ks) * c.scale
        reach = float((torch.einsum("thd,nhd->htn", qs.abs(), ks.abs()) * see).max() * abs(c.scale))
        w = torch.softmax(x.masked_fill(~see, -math.inf), -1)
        res.append((torch.einsum("htn,nhd->thd", w, vs), torch.einsum("htn,nhd->thd", w, vs.abs()), reach))
    return res


def attend_bound(c, s, out, size, reach):
    """What the kernels may be off by.  A score's fp32 sum of D products is off by (D + 4) 2^-23 of sum |q k| at most (the
    tensor cores cut where fp32 rounds: a whole step each), which moves a weight by twice that much relative to the sum of
    all; exp2 adds 2^-22; sums over n positions and their parts another (n + 64) 2^-23.  In bf16 each weight is rounded (half a step of
    itself), and the output once more."""
    n = c.past[s] + c.n(s)
    soft = 2 * ((c.D + 4) * reach + 2) * 2.0 ** -23 + (n + 64) * 2.0 ** -23
    weights = c.half if c.dtype == torch.bfloat16 else 0.0
    return c.half * out.abs() + (weights + soft) * (1 + c.half) * size + 1e-30


def fill_cache(c):
    """Random keys and values of every live position in pools that hold NaN everywhere else.  Per slot [positions][Hk][D]."""
    kp, vp = c.pool(), c.pool()
    ks, vs = [], []
    for s in range(c.B):
        N = c.past[s] + c.n(s)
        k, v = c.rand(N, c.Hk, c.D), c.rand(N, c.Hk, c.D)
        for p0 in range(0, N, c.page):
            page, m = int(c.table[s, p0 // c.page]), min(c.page, N - p0)
            c.rows(kp)[page, :, :m] = k[p0:p0 + m].transpose(0, 1)
            c.rows(vp)[page, :, :m] = v[p0:p0 + m].transpose(0, 1)
        ks.append(k)
        vs.append(v)
    return kp, vp, ks, vs


class Append:
    """What gdn_kv_append does with one head's vector, in 64 bits."""

    def __init__(self, rope, freq, norm, eps, adjacent):
        self.rope, self.freq, self.norm, self.eps, self.adjacent = rope, freq, norm, eps, adjacent

    def __call__(self, x, position):
        """x [heads][D] -> (value, what its error is relative to)."""
        x = x.double()
        if self.norm is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + self.eps) * self.norm.double()
        y, size = x.clone(), x.abs()
        for i in range(self.rope // 2):
            a, b = (2 * i, 2 * i + 1) if self.adjacent else (i, i + self.rope // 2)
            # the angle's part of a turn, exactly: far positions times frequencies
            turn = math.fmod(float(self.freq[i]) * position, 2 * math.pi)
            c, s = math.cos(turn), math.sin(turn)
            y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, a] * s + x[:, b] * c
            size[:, a] = size[:, b] = x[:, a].abs() + x[:, b].abs()
        return y, size


def append_bound(c, y, size):
    """Half a step of the result; 2^-24 of a turn (2 pi 2^-24 radians), cos and sin to 2^-22; a norm's sum of D squares in
    fp32 and a dozen roundings."""
    return c.half * y.abs() + (2 * math.pi * 2.0 ** -24 + 2.0 ** -22 + (c.D + 16) * 2.0 ** -24) * (1 + c.half) * size + 1e-30
