"""The full-attention side of one verify step, as cases to measure.

A hybrid model runs full attention every few layers between its recurrent ones, over the same batch: B requests
("slots") of T new tokens each, a chain, a draft tree or a chunk of a prompt.  What such a layer needs around its
projections, over a key/value cache that is kept in pages:

  append   q and k are normalised per head and rotated by their positions; the rotated k and v of the new tokens go into
           the pages of their slots (after a tree's acceptance: those of the accepted path, at their final places)
  attend   softmax(scale q k^T) v of every new token over what it may see: the slot's past and, of the new tokens, itself
           and those before it (in a tree: its ancestors); with a window, the last positions and a few first ones
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------- the cases

def _case(name, op, slots, tokens, heads, kv_heads, d, page, past, dtype=BF16, ragged=False, form="chain", **more):
    """past: the longest slot's positions before the batch; ragged: slots of other lengths, pasts and token counts."""
    return {"name": name, "op": op, "slots": slots, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "d": d,
            "page": page, "past": past, "dtype": dtype, "ragged": ragged, "form": form, **more}


def _append(name, *sizes, rope, adjacent=False, norm=True, **more):
    return _case(name, "append", *sizes, rope=rope, adjacent=adjacent, norm=norm, **more)


def _attend(name, *sizes, window=0, sinks=0, **more):
    return _case(name, "attend", *sizes, window=window, sinks=sinks, **more)


def listed():
    return [
        # one request, one token: the latency of the call
        _append("append_1x1", 1, 1, 24, 4, 256, 16, 1000, rope=64),
        # the draft trees of 32 slots of different lengths
        _append("append_tree_32x16", 32, 16, 24, 4, 256, 64, 8000, rope=64, ragged=True, form="tree"),
        # a prompt's chunk behind a long beginning, rotated over the whole head in adjacent pairs
        _append("append_prompt_8192", 1, 8192, 32, 8, 128, 128, 20000, rope=128, adjacent=True, norm=False),
        # the accepted paths of eight trees go to their final places
        _append("append_path_8x64_f32", 8, 64, 16, 2, 64, 32, 3000, rope=64, dtype=F32, ragged=True, form="path"),
        # one request decoding one token behind a short context
        _attend("attend_1x1", 1, 1, 24, 4, 256, 16, 1001),
        # one slot's verify of 16 positions
        _attend("attend_1x16", 1, 16, 24, 4, 256, 64, 8185),
        # 32 slots' verify, pasts and counts of all lengths
        _attend("attend_32x16_ragged", 32, 16, 24, 4, 256, 64, 16384, ragged=True),
        # draft trees of 64 nodes
        _attend("attend_tree_8x64", 8, 64, 32, 8, 128, 16, 6000, ragged=True, form="tree"),
        # a few requests decoding behind very long contexts
        _attend("attend_long_4x1", 4, 1, 64, 8, 128, 128, 131000),
        # many slots under a window with a few first tokens that stay visible
        _attend("attend_window_64x2", 64, 2, 40, 8, 64, 32, 20000, ragged=True, window=1024, sinks=4),
        # a prompt's chunk over its own beginning
        _attend("attend_prompt_4096", 1, 4096, 24, 4, 256, 128, 4096),
        # a small model in 32 bits throughout
        _attend("attend_f32_3x5", 3, 5, 8, 2, 64, 16, 333, dtype=F32, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    heads, kv_heads, d = rng.choice([(24, 4, 256), (16, 2, 256), (8, 1, 256), (32, 8, 128), (64, 8, 128), (40, 8, 128),
                                     (16, 16, 128), (28, 4, 128), (8, 2, 64), (40, 8, 64), (12, 12, 64), (64, 4, 64)])
    page, dtype = rng.choice([8, 16, 32, 64, 128, 256]), BF16 if rng.random() < 0.8 else F32
    form = rng.choice(["chain", "chain", "tree", "path", "prompt"] if op == "append" else ["chain", "chain", "tree", "prompt"])
    slots, past = _log_int(rng, 1, 64), _log_int(rng, 1, 65536) - 1
    if form == "prompt":
        slots, tokens = _log_int(rng, 1, 4), _log_int(rng, 65, 4096)
    else:
        tokens = rng.choice([1, 1, 2, 3, 5, 8, 16, 16, 33, 64])
    ragged = slots > 1 and rng.random() < 0.7
    # no more positions in all, scores and bytes than the largest listed cases have
    position = 2 * kv_heads * d * (2 if dtype == BF16 else 4)
    while slots * (past + tokens) * position > 2e9:
        slots, past = (slots + 1) // 2, past if slots > 1 else past // 2
    ceiling = 5e8 if dtype == BF16 else 1e8
    while op == "attend" and slots * tokens * heads * (past + tokens) > ceiling and (past > 64 or slots > 1):
        past, slots = past // 2, max(1, slots // 2) if past <= 2048 else slots
    if slots * tokens > 16384:
        slots = max(1, 16384 // tokens)
    form = "chain" if form == "prompt" else form
    c = _case("", op, slots, tokens, heads, kv_heads, d, page, past, dtype=dtype, ragged=ragged and slots > 1, form=form)
    if op == "append":
        c.update(rope=rng.choice([d, d // 2, d // 4, 0]), adjacent=rng.random() < 0.3, norm=rng.random() < 0.6)
    else:
        windowed = rng.random() < 0.3
        c.update(window=_log_int(rng, 1, 8192) if windowed else 0, sinks=rng.choice([0, 1, 4, 16, 100]) if windowed else 0)
    del c["name"]
    return c


def _lengths(c):
    """What each slot holds before the batch, and how many of its T tokens are real.  Part of the case's size, so not
    drawn: the first slot has the case's sizes, the others follow two sequences that spread evenly."""
    past, length = [c["past"]], [c["tokens"]]
    for s in range(1, c["slots"]):
        past.append(int(c["past"] * ((s * 0.6180339887) % 1.0)) if c["ragged"] else c["past"])
        length.append(1 + int(c["tokens"] * ((s * 0.7548776662) % 1.0)) if c["ragged"] else c["tokens"])
    return past, length


# ------------------------------------------------------------------------------------------- inputs (both sides)

def prepare(case, seed):
    """Pools of pages in a random order, each slot's page table (-1 behind its last page), and the batch's rows."""
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dtype = _TORCH[c["dtype"]]
    rand = lambda std, *shape: (torch.randn(shape, generator=g, device=dev) * std).to(dtype)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    B, T, H, Hk, D, P = c["slots"], c["tokens"], c["heads"], c["kv_heads"], c["d"], c["page"]
    past, length = _lengths(c)
    pages = [-(-(p + T) // P) for p in past]
    width, total = max(pages), sum(pages) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    count = i32(pages)
    first = (count.cumsum(0) - count).unsqueeze(1)
    at = torch.arange(width, device=dev).unsqueeze(0)
    table = torch.where(at < count.unsqueeze(1), order[(first + at).clamp(max=total - 1)], -1).to(torch.int32)
    pool = lambda: torch.randn((total, Hk, P, D), generator=g, device=dev, dtype=dtype)  # noqa: E731
    s = {"case": c, "table": table, "past": i32(past), "length": i32(length) if c["ragged"] else None, "n_pages": total,
         "k_pool": pool(), "v_pool": pool(), "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    node = torch.arange(T, device=dev)
    if c["form"] == "tree":
        # a node's parent lies among the eight before it, most often near; node 0 is the last committed token
        back = 1 + (torch.rand((B, T), generator=g, device=dev) ** 2 * 8).long()
        parent = (node - back).clamp(min=0)
        parent[:, 0] = -1
        s["parent"] = parent.to(torch.int32).contiguous()
    elif c["form"] == "path":
        # an accepted path: node 0, then nodes in rising order, about one in three
        on = torch.rand((B, T), generator=g, device=dev) < 0.35
        on[:, 0] = True
        path = torch.sort(torch.where(on, node, T), dim=1).values
        s["path"] = torch.where(path < T, path, -1).to(torch.int32)
    if c["op"] == "append":
        s["rows"] = rand(1.0, B * T, (H + 2 * Hk) * D)         # a row of the fused projection: q, then k, then v
        s["q_out"] = torch.zeros((B, T, H, D), dtype=dtype, device=dev)
        s["q_norm"] = 0.5 + torch.rand(D, generator=g, device=dev)
        s["k_norm"] = 0.5 + torch.rand(D, generator=g, device=dev)
        half = c["rope"] // 2
        s["freq"] = (1e7 ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(half, 1))).float()
    else:
        s["q"] = rand(1.5, B, T, H, D)
        s["out"] = torch.zeros((B, T, H, D), dtype=dtype, device=dev)
    return s


# ------------------------------------------------------------------------------------------------ the plain forms

def _ancestors(parent):
    """[slot][node][node']: whether node' is the node itself or an ancestor of it."""
    T = parent.shape[1]
    at = torch.arange(T, device=parent.device)
    step = (parent.long().unsqueeze(2) == at).double() + torch.eye(T, dtype=torch.float64, device=parent.device)
    return torch.matrix_power(step, T) > 0


def _live(s):
    T = s["case"]["tokens"]
    at = torch.arange(T, device=s["table"].device)
    return at < (s["length"].unsqueeze(1) if s["length"] is not None else torch.full_like(s["past"], T).unsqueeze(1))


def _rotate(s, x, norm, position):
    """x [B][T][heads][D] in 32 bits; the angles in 64: far positions times frequencies lose their turns in 32."""
    c = s["case"]
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * norm
    n = c["rope"]
    angle = position.double().unsqueeze(2) * s["freq"].double()
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    turned, rest = x[..., :n], x[..., n:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if c["adjacent"] else (turned[..., :n // 2], turned[..., n // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((a, b), -1).flatten(-2) if c["adjacent"] else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _plain_append(s):
    c = s["case"]
    B, T, H, Hk, D, P = c["slots"], c["tokens"], c["heads"], c["kv_heads"], c["d"], c["page"]
    q, k, v = s["rows"].reshape(B, T, H + 2 * Hk, D).split((H, Hk, Hk), dim=2)
    at = torch.arange(T, device=q.device).expand(B, T)
    live, depth = _live(s), at
    if c["form"] == "tree":
        depth = _ancestors(s["parent"]).sum(2) - 1
    elif c["form"] == "path":
        live = live & (s["path"] >= 0)
        row = s["path"].long().clamp(min=0)[:, :, None, None].expand(B, T, Hk, D)
        k, v = k.gather(1, row), v.gather(1, row)
    place = s["past"].long().unsqueeze(1) + at
    position = s["past"].long().unsqueeze(1) + depth
    k = _rotate(s, k.float(), s["k_norm"], position).to(q.dtype)
    page = s["table"].long().gather(1, (place // P).clamp(max=s["table"].shape[1] - 1))
    # rows that are not real go nowhere: a page of their own behind the pool
    page = torch.where(live, page, s["n_pages"])
    outs = {}
    for name, rows in (("k", k), ("v", v)):
        pool = s[name + "_pool"]
        wide = torch.cat((pool, pool[:1]))
        wide[page, :, place % P] = rows
        pool.copy_(wide[:-1])
        outs[name] = pool
    if c["form"] != "path":
        q = _rotate(s, q.float(), s["q_norm"], position).to(q.dtype)
        outs["q"] = torch.where(live[:, :, None, None], q, s["q_out"])
    return outs


def _plain_attend(s):
    c = s["case"]
    B, T, H, Hk, D, P = c["slots"], c["tokens"], c["heads"], c["kv_heads"], c["d"], c["page"]
    G, N = H // Hk, s["table"].shape[1] * P
    page = s["table"].long().clamp(min=0)
    gather = lambda pool: pool[page].transpose(1, 2).reshape(B, Hk, N, D).float()  # noqa: E731
    past, at = s["past"].long().view(B, 1, 1), torch.arange(T, device=page.device)
    live = _live(s)
    if c["form"] == "tree":
        seen = _ancestors(s["parent"])
        position = past[:, 0] + seen.sum(2) - 1                                    # [B][T]
        key = torch.arange(N, device=page.device).expand(B, 1, N)
        node = (key - past).clamp(0, T - 1)
        among = torch.cat((seen, seen[:, :, :1] & False), 2).gather(2, node.expand(B, T, N)) & (key < past + T)
        visible = (key < past) | among
        where = torch.where(key < past, key, past + position.sub(past[:, 0]).unsqueeze(1).gather(2, node))
    else:
        position = past[:, 0] + at
        where = torch.arange(N, device=page.device).expand(B, 1, N)
        visible = where <= position.unsqueeze(2)
    if c["window"]:
        visible = visible & ((where > position.unsqueeze(2) - c["window"]) | (where < c["sinks"]))
    # nothing but zeros where a slot holds nothing
    held = (torch.arange(N, device=page.device) < past[:, :, 0] + T).view(B, 1, N, 1)
    k = torch.where(held, gather(s["k_pool"]), 0.0)
    q = s["q"].float().reshape(B, T, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * T, D)
    score = ((q * D ** -0.5) @ k.transpose(2, 3)).reshape(B, Hk, G, T, N)
    del k
    score.masked_fill_(~visible.view(B, 1, 1, T, N), float("-inf"))
    score -= score.amax(-1, keepdim=True)
    weight = score.exp_()
    total = weight.sum(-1, keepdim=True)
    v = torch.where(held, gather(s["v_pool"]), 0.0)
    out = (weight.reshape(B, Hk, G * T, N) @ v).reshape(B, Hk, G, T, D) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(B, T, H, D).to(s["q"].dtype)
    return {"out": torch.where(live[:, :, None, None], out, s["out"])}


# ---------------------------------------------------------------------------------------- the framework's own calls

def _plan(s):
    import gated_deltanet_verify_gb300 as gdn
    if "plan" not in s:
        c = s["case"]
        dims = gdn.make_attn_dims(c["slots"], c["tokens"], c["heads"], c["kv_heads"], c["d"], c["page"], s["n_pages"],
                                  s["table"].shape[1], dtype=gdn.GDN_BF16 if c["dtype"] == BF16 else gdn.GDN_F32)
        cache = gdn.kv_cache(s["k_pool"], s["v_pool"], s["table"], s["past"])
        if c["op"] == "append":
            norms = (s["q_norm"], s["k_norm"]) if c["norm"] else (None, None)
            more = gdn.qk_params(c["rope"], s["freq"] if c["rope"] else None, *norms, norm_eps=EPS, adjacent=c["adjacent"])
        else:
            size = gdn.gdn_attend_workspace_bytes(dims)
            more = (gdn.attn_params(c["d"] ** -0.5, c["window"], c["sinks"]),
                    torch.empty(size, dtype=torch.uint8, device="cuda"), size)
        s["plan"] = (gdn, dims, cache, more)
    return s["plan"]


def _own_append(s):
    gdn, dims, cache, params = _plan(s)
    c, rows = s["case"], s["rows"]
    ld, hd, kd = rows.shape[1], c["heads"] * c["d"], c["kv_heads"] * c["d"]
    path = c["form"] == "path"
    gdn.gdn_kv_append(dims, cache, params, None if path else rows, rows[:, hd:], rows[:, hd + kd:], ld, ld, ld,
                      None if path else s["q_out"], d_length=s["length"], d_parent=s.get("parent"),
                      d_path=s.get("path"), d_status=s["status"])
    outs = {"k": s["k_pool"], "v": s["v_pool"]}
    if not path:
        outs["q"] = s["q_out"]
    return outs


def _own_attend(s):
    gdn, dims, cache, (params, space, size) = _plan(s)
    gdn.gdn_attend(dims, cache, params, s["q"], s["out"], space, size, d_length=s["length"], d_parent=s.get("parent"),
                   d_status=s["status"])
    return {"out": s["out"]}


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_attend(state) if own else _plain_attend(state)


def work(case):
    c = case
    past, length = _lengths(c)
    H, Hk, D, size = c["heads"], c["kv_heads"], c["d"], 2 if c["dtype"] == BF16 else 4
    rows = sum(length)
    if c["op"] == "append":
        # every real row read and written once; a norm and a rotation for each element of q and k
        moved = (2 * Hk if c["form"] == "path" else H + 2 * Hk) * D * rows
        return {"bytes": 2 * size * moved + 8 * c["slots"], "flops": 8.0 * rows * (H + Hk) * D}
    pairs = keys = 0
    for p, n in zip(past, length):
        reach = c["window"] or p + n
        for t in range(n):
            # of a tree's nodes, itself alone: its ancestors are not known from the sizes
            seen = p + 1 if c["form"] == "tree" else p + t + 1
            pairs += min(seen, reach + min(c["sinks"], max(0, seen - reach)))
        low = max(0, p + 1 - reach)
        keys += p + n - low + min(c["sinks"], low)
    return {"bytes": size * D * (2 * Hk * keys + 2 * H * rows) + 8 * c["slots"], "flops": 4.0 * H * D * pairs}


# -------------------------------------------------------------------------------- the definition, in 64 bits, apart

def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _exact_append(s):
    c = s["case"]
    B, T, H, Hk, D, P = c["slots"], c["tokens"], c["heads"], c["kv_heads"], c["d"], c["page"]
    past, length = _lengths(c)
    table, n = s["table"].tolist(), c["rope"]
    rows = s["rows"].double().reshape(B, T, H + 2 * Hk, D)
    k_pool, v_pool, q_out = s["k_pool"].double(), s["v_pool"].double(), s["q_out"].double()
    freq = s["freq"].double()

    def turned(x, weight, positions):
        """A pair as a complex number, turned by multiplication with e^(i angle)."""
        if c["norm"]:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
        if not n:
            return x
        angle = torch.tensor(positions, dtype=torch.float64, device=x.device)[:, None] * freq
        unit = torch.polar(torch.ones_like(angle), angle)[:, None]
        pairs = x[..., :n].unflatten(-1, (n // 2, 2) if c["adjacent"] else (2, n // 2))
        if not c["adjacent"]:
            pairs = pairs.transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        if not c["adjacent"]:
            pairs = pairs.transpose(-1, -2)
        return torch.cat((pairs.flatten(-2), x[..., n:]), -1)

    for b in range(B):
        m = length[b]
        source = list(range(m))
        depth = source
        if c["form"] == "tree":
            depth = _depths(s["parent"][b, :m].tolist())
        elif c["form"] == "path":
            source = [i for i in s["path"][b, :m].tolist() if i >= 0]
            depth = list(range(len(source)))
        spot = [past[b] + d for d in depth]
        x = rows[b, source]
        k = turned(x[:, H:H + Hk], s["k_norm"], spot)
        pages = torch.tensor([table[b][(past[b] + i) // P] for i in range(len(source))], device=x.device)
        inside = torch.tensor([(past[b] + i) % P for i in range(len(source))], device=x.device)
        k_pool[pages, :, inside], v_pool[pages, :, inside] = k, x[:, H + Hk:]
        if c["form"] != "path":
            q_out[b, :m] = turned(x[:, :H], s["q_norm"], spot)
    outs = {"k": k_pool, "v": v_pool}
    if c["form"] != "path":
        outs["q"] = q_out
    return outs


def _exact_attend(s):
    c = s["case"]
    if work(c)["flops"] > 3e12:
        return None
    T, H, Hk, D, P = c["tokens"], c["heads"], c["kv_heads"], c["d"], c["page"]
    past, length = _lengths(c)
    out = s["out"].double()
    for b in range(c["slots"]):
        p, n = past[b], length[b]
        spot = list(range(p, p + n))
        if c["form"] == "tree":
            parents = s["parent"][b, :n].tolist()
            spot = [p + d for d in _depths(parents)]
        where = torch.tensor(list(range(p)) + spot, device=out.device)
        mine = where[p:, None]
        may = torch.ones((n, p + n), dtype=torch.bool, device=out.device)
        if c["form"] == "tree":
            lines = torch.zeros((n, n), dtype=torch.bool)
            for t, u in enumerate(parents):
                if u >= 0:
                    lines[t] = lines[u]
                lines[t, t] = True
            may[:, p:] = lines.to(out.device)
        else:
            may[:, p:] = torch.ones((n, n), dtype=torch.bool, device=out.device).tril()
        if c["window"]:
            may &= (mine - where < c["window"]) | (where < c["sinks"])
        ids = s["table"][b, :-(-(p + n) // P)].long()
        for h in range(Hk):
            k = s["k_pool"][ids, h].reshape(-1, D)[:p + n].double()
            v = s["v_pool"][ids, h].reshape(-1, D)[:p + n].double()
            for j in range(h * (H // Hk), (h + 1) * (H // Hk)):
                x = torch.einsum("td,nd->tn", s["q"][b, :n, j].double(), k) / math.sqrt(D)
                out[b, :n, j] = torch.softmax(x.masked_fill(~may, -math.inf), 1) @ v
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
