"""The operators around one verify step that differ from slot to slot, as cases to measure.

A verify step serves a batch of requests ("slots").  On its way in every slot may carry a low-rank adapter of its
own beside the shared projections; on its way out every slot's positions are sampled with that slot's parameters,
and the sampled tokens decide how many of the drafted tokens the slot keeps, which is what a rollback takes:

  lora_in, lora_out   act = x W^T + scale_a (x A_a^T) B_a^T, adapter a by slot (-1: none)
  sample              temperature, top-k, top-p and min-p, from given uniforms
  accept, accept_tree the longest drafted prefix (path of the draft tree) that agrees with the sampled tokens
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_TORCH = {F32: torch.float32, BF16: torch.bfloat16}


# ---------------------------------------------------------------------------------------------------- the cases

def _sample(name, slots, tokens, vocab, dtype, filters, masked=False, pad=0):
    return {"name": name, "op": "sample", "slots": slots, "tokens": tokens, "vocab": vocab, "dtype": dtype,
            "filters": filters, "masked": masked, "pad": pad}


def _accept(name, op, slots, tokens, ragged):
    return {"name": name, "op": op, "slots": slots, "tokens": tokens, "ragged": ragged}


def _lora(name, op, slots, tokens, qk_heads, v_heads, d, embd, rank, adapters):
    return {"name": name, "op": op, "slots": slots, "tokens": tokens, "qk_heads": qk_heads, "v_heads": v_heads,
            "d": d, "embd": embd, "rank": rank, "adapters": adapters}


def listed():
    return [
        # one request decoding one token: the latency of the call
        _sample("sample_one_row", 1, 1, 32768, F32, "all"),
        # the 16 positions of one slot's verify, nucleus sampling over a large vocabulary
        _sample("sample_verify_16", 1, 16, 131072, BF16, "top_p"),
        # eight slots, no filter; an odd vocabulary, so rows start on any 4-byte boundary
        _sample("sample_8x16_odd", 8, 16, 100003, F32, "none"),
        # sixteen requests, each with its own filters, some greedy, some under a grammar's mask (one allows nothing)
        _sample("sample_16x16_mixed", 16, 16, 200000, F32, "mixed", masked=True),
        # the acceptance of one ordinary batch, of many ragged slots, of one draft tree and of many
        _accept("accept_8x16", "accept", 8, 16, False),
        _accept("accept_1024x64_ragged", "accept", 1024, 64, True),
        _accept("accept_tree_1x16", "accept_tree", 1, 16, False),
        _accept("accept_tree_256x64", "accept_tree", 256, 64, True),
        # the layer's input projection for one slot with an adapter, and for 32 slots with one each
        _lora("lora_in_1x16", "lora_in", 1, 16, 16, 48, 128, 5120, 16, 8),
        _lora("lora_in_32x16", "lora_in", 32, 16, 16, 48, 128, 5120, 16, 48),
        # the output projection with a higher rank
        _lora("lora_out_8x16_r64", "lora_out", 8, 16, 16, 48, 128, 5120, 64, 12),
        # a small layer with ragged sizes
        _lora("lora_in_small", "lora_in", 3, 5, 2, 8, 64, 264, 8, 3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "accept", "accept_tree", "lora_in", "lora_in", "lora_out"])
    if op == "sample":
        slots, tokens = _log_int(rng, 1, 32), rng.choice([1, 1, 2, 5, 8, 16])
        vocab = _log_int(rng, 1000, 200000)
        while slots * tokens > 256:
            slots = (slots + 1) // 2
        c = _sample("", slots, tokens, vocab, rng.choice([F32, BF16]),
                    rng.choice(["none", "top_k", "top_p", "min_p", "all", "mixed", "greedy"]), rng.random() < 0.3,
                    rng.choice([0, 0, 1, 8, 61]))
    elif op in ("accept", "accept_tree"):
        c = _accept("", op, _log_int(rng, 1, 1024 if op == "accept" else 256), rng.randint(1, 64), rng.random() < 0.5)
    else:
        v_heads, group = rng.choice([(8, 1), (8, 2), (16, 2), (24, 3), (48, 3)])
        slots = _log_int(rng, 1, 32)
        c = _lora("", op, slots, rng.randint(1, 16), v_heads // group, v_heads, rng.choice([32, 64, 128]),
                  8 * _log_int(rng, 8, 640), rng.choice([8, 16, 24, 32, 64, 128]), _log_int(rng, 1, 48))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------- inputs (both sides)

def _gen(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def _prepare_sample(c, seed):
    """Logits with a Zipf-like head (as a language model's) under noise; parameters per slot; one uniform per row."""
    g, dev = _gen(seed, "cuda"), "cuda"
    B, T, V = c["slots"], c["tokens"], c["vocab"]
    rows, ld = B * T, c["vocab"] + c["pad"]
    noise = torch.randn((rows, ld), generator=g, device=dev)
    shift = torch.randint(0, V, (rows, 1), generator=g, device=dev)
    # a rank for every token, another order in every row: multiplication by a number prime to the vocabulary
    step = next(p for p in (7919, 104729, 1299709, 15485863) if math.gcd(p, V) == 1)
    rank = (torch.arange(ld, device=dev).unsqueeze(0) * step + shift) % V
    full = 6.0 + 1.2 * noise - 1.1 * torch.log1p(rank.float())
    del noise, rank
    kind = torch.arange(B, device=dev) % 8
    if c["masked"]:
        # a grammar's mask over every third slot: 2 tokens in 100 stay; the batch's last position allows none
        allowed = torch.rand((rows, ld), generator=g, device=dev) < 0.02
        slot = torch.arange(rows, device=dev) // T
        under = (slot % 3 == 0).unsqueeze(1)
        full = torch.where(under & ~allowed, float("-inf"), full)
        last = torch.zeros(rows, dtype=torch.bool, device=dev)
        last[-1] = B > 1
        full = full.masked_fill(last.unsqueeze(1), float("-inf"))
    logits = full.to(_TORCH[c["dtype"]])
    del full
    uni = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=g, device=dev)  # noqa: E731
    temp, top_p, min_p = uni(0.6, 1.3), uni(0.8, 0.98), uni(0.01, 0.1)
    top_k = torch.randint(1, 101, (B,), generator=g, device=dev, dtype=torch.int32)
    f = c["filters"]
    if f == "mixed":
        temp = torch.where(kind == 0, 0.0, temp)
        top_k = torch.where((kind == 1) | (kind == 4) | (kind == 7), top_k, 0)
        top_p = torch.where((kind == 2) | (kind == 4) | (kind == 6) | (kind == 7), top_p, 1.0)
        min_p = torch.where((kind == 3) | (kind == 6) | (kind == 7), min_p, 0.0)
    elif f != "all":
        temp = torch.zeros_like(temp) if f == "greedy" else temp
        top_k = top_k if f == "top_k" else torch.zeros_like(top_k)
        top_p = top_p if f == "top_p" else torch.ones_like(top_p)
        min_p = min_p if f == "min_p" else torch.zeros_like(min_p)
    return {"case": c, "logits": logits, "temp": temp, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "u": torch.rand((B, T), generator=g, device=dev),
            "tokens": torch.empty((B, T), dtype=torch.int32, device=dev),
            "logprob": torch.empty((B, T), dtype=torch.float32, device=dev)}


def _prepare_accept(c, seed):
    """Sampled tokens, and drafts that agree with them four times in five; in a tree a node's children carry
    distinct guesses, one of them mostly the sampled one."""
    g, dev = _gen(seed, "cuda"), "cuda"
    B, T = c["slots"], c["tokens"]
    tokens = torch.randint(0, 200000, (B, T), generator=g, device=dev, dtype=torch.int32)
    miss = torch.rand((B, T), generator=g, device=dev) < 0.2
    wrong = torch.randint(0, 200000, (B, T), generator=g, device=dev, dtype=torch.int32)
    length = (torch.randint(1, T + 1, (B,), generator=g, device=dev, dtype=torch.int32) if c["ragged"]
              else torch.full((B,), T, dtype=torch.int32, device=dev))
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": c, "tokens": tokens, "length": length, "place": i32(B), "next": i32(B), "emit": i32(B, T)}
    at = torch.arange(T, device=dev)
    if c["op"] == "accept":
        parent = (at - 1).expand(B, T)
    else:
        # a node's parent lies among the eight before it, most often near
        back = 1 + (torch.rand((B, T), generator=g, device=dev) ** 2 * 8).long()
        parent = (at - back).clamp(min=0)
        parent[:, 0] = -1
        s["parent"], s["path"] = parent.to(torch.int32).contiguous(), i32(B, T)
    right = tokens.gather(1, parent.clamp(min=0))
    s["draft"] = torch.where(miss, wrong, right)
    return s


def _shape(c):
    conv = 2 * c["qk_heads"] * c["d"] + c["v_heads"] * c["d"]
    value = c["v_heads"] * c["d"]
    n_in = conv + value + 2 * c["v_heads"]
    return (n_in, c["embd"]) if c["op"] == "lora_in" else (c["embd"], value)     # output and input columns


def _prepare_lora(c, seed):
    g, dev = _gen(seed, "cuda"), "cuda"
    N, K = _shape(c)
    M, r, n = c["slots"] * c["tokens"], c["rank"], c["adapters"]
    rand = lambda std, *shape: (torch.randn(shape, generator=g, device=dev) * std).to(torch.bfloat16)  # noqa: E731
    ids = torch.randint(0, n, (c["slots"],), generator=g, device=dev, dtype=torch.int32)
    if c["slots"] > 2:
        ids = torch.where(torch.rand(c["slots"], generator=g, device=dev) < 0.125, -1, ids).to(torch.int32)
    other = (c["embd"], c["v_heads"] * c["d"]) if c["op"] == "lora_in" else (_in_columns(c), c["embd"])
    return {"case": c, "x": rand(1.0, M, K), "w": rand(K ** -0.5, N, K), "a": rand(K ** -0.5, n, r, K),
            "b": rand(0.5 * r ** -0.5, n, N, r), "scale": 0.5 + torch.rand(n, generator=g, device=dev), "ids": ids,
            "y": torch.empty((M, N), dtype=torch.bfloat16, device=dev),
            "other": torch.zeros(other, dtype=torch.bfloat16, device=dev)}   # the layer's other projection


def _in_columns(c):
    return 2 * c["qk_heads"] * c["d"] + 2 * c["v_heads"] * c["d"] + 2 * c["v_heads"]


def prepare(case, seed):
    if case["op"] == "sample":
        s = _prepare_sample(case, seed)
    elif case["op"] in ("accept", "accept_tree"):
        s = _prepare_accept(case, seed)
    else:
        s = _prepare_lora(case, seed)
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ the plain forms

def _plain_sample(s):
    c = s["case"]
    B, T, V = c["slots"], c["tokens"], c["vocab"]
    # 64 bits: a token is chosen where a sum over the vocabulary passes a border
    logits = s["logits"][:, :V].double()
    logits = torch.where(logits.isnan(), float("-inf"), logits)
    row = lambda v: v.repeat_interleave(T).unsqueeze(1)  # noqa: E731
    temp, top_k, top_p, min_p = row(s["temp"]).double(), row(s["top_k"]), row(s["top_p"]).double(), row(s["min_p"]).double()
    best = logits.amax(1, keepdim=True)
    none = best == float("-inf")
    greedy = temp == 0
    x = torch.where(logits == best, 0.0, (logits - best) / torch.where(greedy, 1.0, temp))
    weight = torch.exp(x)
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices
    del logits
    down = weight.gather(1, order)
    place = torch.arange(V, device=x.device).unsqueeze(0)
    keep = torch.where(greedy, place < 1, (top_k <= 0) | (place < top_k))
    down = down * keep
    before = down.cumsum(1) - down
    keep &= (top_p >= 1) | (before < top_p * down.sum(1, keepdim=True)) | (place < 1)
    keep &= (min_p <= 0) | (down >= min_p)
    del down, before
    kept = weight * torch.zeros_like(keep).scatter_(1, order, keep)
    del weight, order, keep
    total = kept.sum(1, keepdim=True)
    u = s["u"].reshape(-1, 1).double()
    token = (kept.cumsum(1) <= u * total).sum(1, keepdim=True)
    # past the end by a rounding of the last sum: the last token that is kept
    token = torch.minimum(token, torch.where(kept > 0, place, 0).amax(1, keepdim=True))
    logprob = torch.where(none, float("-inf"), x.gather(1, token) - total.log())
    token = torch.where(none, -1, token)
    return {"tokens": token.reshape(B, T).to(torch.int32), "logprob": logprob.reshape(B, T).float()}


def _plain_accept(s):
    T = s["case"]["tokens"]
    tokens, at = s["tokens"], torch.arange(T, device=s["tokens"].device)
    same = (s["draft"][:, 1:] == tokens[:, :-1]) & (tokens[:, :-1] >= 0) & (at[1:] < s["length"].unsqueeze(1))
    n = same.long().cumprod(1).sum(1, keepdim=True)
    i32 = lambda v: v.to(torch.int32)  # noqa: E731
    return {"trim": i32(T - 1 - n[:, 0]), "next": tokens.gather(1, n)[:, 0],
            "emit": i32(torch.where(at <= n, tokens, -1))}


def _plain_accept_tree(s):
    T = s["case"]["tokens"]
    tokens, draft, parent = s["tokens"], s["draft"], s["parent"].long()
    at = torch.arange(T, device=tokens.device)
    sampled = tokens.gather(1, parent.clamp(min=0))
    same = (draft == sampled) & (sampled >= 0) & (parent >= 0) & (at < s["length"].unsqueeze(1))
    # of a node's children with the same token the first one counts
    twin = (parent.unsqueeze(2) == parent.unsqueeze(1)) & (draft.unsqueeze(2) == draft.unsqueeze(1)) & (at.unsqueeze(1) > at)
    same &= ~twin.any(2)
    # edges that are followed, and what node 0 reaches over them
    edge = (parent.unsqueeze(2) == at) & same.unsqueeze(2)                       # [slot][child][parent]
    step = edge.transpose(1, 2).float() + torch.eye(T, device=tokens.device)
    reached = torch.matrix_power(step.clamp(max=1).double(), max(1, T))[:, 0] > 0
    last = torch.where(reached, at, 0).amax(1, keepdim=True)
    path = torch.sort(torch.where(reached, at, T), dim=1).values
    live = path < T
    path = path.clamp(max=T - 1)
    i32 = lambda v: v.to(torch.int32)  # noqa: E731
    return {"accept": i32(last[:, 0]), "next": tokens.gather(1, last)[:, 0],
            "emit": i32(torch.where(live, tokens.gather(1, path), -1)), "path": i32(torch.where(live, path, -1))}


def _plain_lora(s):
    c = s["case"]
    x, ids = s["x"].float(), s["ids"].long()
    y = x @ s["w"].float().T
    used = ids.clamp(min=0)
    scale = torch.where(ids >= 0, s["scale"][used], 0.0).reshape(-1, 1, 1)
    h = x.reshape(c["slots"], c["tokens"], -1) @ s["a"][used].float().transpose(1, 2)
    y += ((h * scale) @ s["b"][used].float().transpose(1, 2)).reshape(y.shape)
    return {"y": y.to(torch.bfloat16)}


# ---------------------------------------------------------------------------------------- the framework's own calls

def _dims(c):
    import gated_deltanet_verify_gb300 as gdn
    return gdn.make_dims(c["slots"], c.get("qk_heads", 1), c.get("v_heads", 1), c.get("d", 32), c.get("d", 32), c["tokens"])


def _own_sample(s):
    import gated_deltanet_verify_gb300 as gdn
    c = s["case"]
    if "plan" not in s:
        s["plan"] = (gdn.make_sample_dims(c["slots"], c["tokens"], c["vocab"], ld=c["vocab"] + c["pad"],
                                          dtype=gdn.GDN_BF16 if c["dtype"] == BF16 else gdn.GDN_F32),
                     gdn.sample_params(s["temp"], s["top_k"], s["top_p"], s["min_p"]))
    dims, params = s["plan"]
    gdn.gdn_sample(dims, params, s["logits"], s["u"], s["tokens"], s["logprob"], s["status"])
    return {"tokens": s["tokens"], "logprob": s["logprob"]}


def _own_accept(s):
    import gated_deltanet_verify_gb300 as gdn
    if "plan" not in s:
        s["plan"] = _dims(s["case"])
    gdn.gdn_accept(s["plan"], s["draft"], s["tokens"], s["length"], s["place"], s["next"], s["emit"], s["status"])
    return {"trim": s["place"], "next": s["next"], "emit": s["emit"]}


def _own_accept_tree(s):
    import gated_deltanet_verify_gb300 as gdn
    if "plan" not in s:
        s["plan"] = _dims(s["case"])
    gdn.gdn_accept_tree(s["plan"], s["parent"], s["draft"], s["tokens"], s["length"], s["place"], s["next"], s["emit"],
                        s["path"], s["status"])
    return {"accept": s["place"], "next": s["next"], "emit": s["emit"], "path": s["path"]}


def _own_lora(s):
    import gated_deltanet_verify_gb300 as gdn
    c = s["case"]
    if "plan" not in s:
        dims = _dims(c)
        w = (s["w"], s["other"]) if c["op"] == "lora_in" else (s["other"], s["w"])
        size = gdn.gdn_lora_workspace_bytes(dims, c["rank"])
        s["plan"] = (dims, gdn.proj_weights(c["embd"], *w),
                     gdn.lora(c["adapters"], c["rank"], s["a"], s["b"], s["scale"]),
                     torch.empty(size, dtype=torch.uint8, device="cuda"), size)
    dims, w, lora, space, size = s["plan"]
    call = gdn.gdn_project_in_lora if c["op"] == "lora_in" else gdn.gdn_project_out_lora
    call(dims, w, lora, s["ids"], s["x"], s["y"], space, size, s["status"])
    return {"y": s["y"]}


def run(state):
    op = state["case"]["op"]
    if op == "sample":
        return _own_sample(state) if own else _plain_sample(state)
    if op == "accept":
        return _own_accept(state) if own else _plain_accept(state)
    if op == "accept_tree":
        return _own_accept_tree(state) if own else _plain_accept_tree(state)
    return _own_lora(state) if own else _plain_lora(state)


def work(case):
    c = case
    if c["op"] == "sample":
        rows = c["slots"] * c["tokens"]
        # every logit read once; a difference, a product, an exponential and a sum for each
        return {"bytes": rows * (c["vocab"] * (2 if c["dtype"] == BF16 else 4) + 12) + 16 * c["slots"],
                "flops": 4.0 * rows * c["vocab"]}
    if c["op"] in ("accept", "accept_tree"):
        tensors = 3 if c["op"] == "accept" else 5          # drafts, tokens, emitted tokens; parents and the path
        return {"bytes": 4 * c["slots"] * (tensors * c["tokens"] + 3), "flops": c["slots"] * c["tokens"]}
    N, K = _shape(c)
    M, r = c["slots"] * c["tokens"], c["rank"]
    used = min(c["slots"], c["adapters"])
    return {"bytes": 2 * (M * K + N * K + M * N + used * r * (N + K)) + 4 * c["slots"],
            "flops": 2.0 * M * (N * K + r * (N + K))}


# -------------------------------------------------------------------------------- the definition, in 64 bits, apart

def _exact_sample(s):
    import numpy as np
    c = s["case"]
    B, T, V = c["slots"], c["tokens"], c["vocab"]
    if B * T * V > 60_000_000:
        return None
    get = lambda k: s[k].double().cpu().numpy()  # noqa: E731
    temp, top_k, top_p, min_p, u = get("temp"), get("top_k"), get("top_p"), get("min_p"), get("u")
    tokens, logprob = np.full((B, T), -1, np.int32), np.full((B, T), -np.inf)
    for b in range(B):
        for t in range(T):
            v = s["logits"][b * T + t, :V].double().cpu().numpy()
            live = np.flatnonzero(v > -np.inf)
            if not live.size:
                continue
            if temp[b] == 0:
                tokens[b, t], logprob[b, t] = np.argmax(np.where(np.isnan(v), -np.inf, v)), 0.0
                continue
            # most likely first, the lower index first among equals
            live = live[np.argsort(-v[live], kind="stable")]
            p = np.exp((v[live] - v[live[0]]) / temp[b])
            n = live.size
            if top_k[b] > 0:
                n = min(n, int(top_k[b]))
            if top_p[b] < 1:
                part = np.cumsum(p[:n])
                n = min(n, 1 + int(np.count_nonzero(part < top_p[b] * part[-1])))
            if min_p[b] > 0:
                n = min(n, int(np.count_nonzero(p >= min_p[b])))
            chosen = np.argsort(live[:n])
            part = np.cumsum(p[:n][chosen])
            i = min(n - 1, int(np.searchsorted(part, u[b, t] * part[-1], side="right")))
            tokens[b, t], logprob[b, t] = live[chosen[i]], math.log(p[chosen[i]] / part[-1])
    return {"tokens": torch.from_numpy(tokens), "logprob": torch.from_numpy(logprob)}


def _exact_lora(s):
    x, y = s["x"].double(), s["x"].double() @ s["w"].double().T
    T = s["case"]["tokens"]
    for b, i in enumerate(s["ids"].tolist()):
        if i >= 0:
            rows = slice(b * T, (b + 1) * T)
            y[rows] += s["scale"][i].double() * (x[rows] @ s["a"][i].double().T @ s["b"][i].double().T)
    return {"y": y}


def exact(case, seed):
    if case["op"] == "sample":
        return _exact_sample(prepare(case, seed))
    if case["op"] in ("lora_in", "lora_out"):
        return _exact_lora(prepare(case, seed))
    return None       # whole numbers alone
