"""The full-attention side of a hybrid model's verify step beside its recurrent side: a draft tree runs through both, the
acceptance moves both, and the next step goes on from there."""
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.attn_ref import Case, attend_bound, attend_ref, fill_cache, line

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


B, T, H, HK, D, PAGE, ROPE = 3, 16, 24, 4, 256, 16, 64
GB = dict(Hk=2, Hv=8, dk=64, dv=64)                        # the recurrent layer's heads


class Attention:
    """One layer's cache, and the buffers of one batch."""

    def __init__(self, past, seed):
        c = self.c = Case(T, H, HK, D, PAGE, [p + 3 * T for p in past], seed=seed)       # pages for some steps to come
        c.pages()
        c.past = list(past)
        g = torch.Generator().manual_seed(seed)
        kp, vp, self.ks, self.vs = self.fill()
        self.k, self.v, self.table = kp.cuda(), vp.cuda(), c.table.cuda()
        self.past = torch.tensor(past, dtype=torch.int32, device="cuda")
        freq = (1e6 ** (-torch.arange(ROPE // 2, dtype=torch.float64) / (ROPE // 2))).float().cuda()
        w = [(0.5 + torch.rand(D, generator=g)).cuda() for _ in range(2)]
        self.params = gdn.qk_params(ROPE, freq, *w)
        self.dims = c.dims()
        self.space_bytes = gdn.gdn_attend_workspace_bytes(self.dims)
        self.space = torch.empty(self.space_bytes, dtype=torch.uint8, device="cuda")
        self.q = torch.zeros((B, T, H, D), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fill(self):
        """Positions 0 .. past of every slot, without the batch."""
        c, keep = self.c, self.c.length
        c.length = [0] * B
        r = fill_cache(c)
        c.length = keep
        return r

    def cache(self):
        return gdn.kv_cache(self.k, self.v, self.table, self.past)

    def append(self, rows, **kw):
        flat = rows.view(-1)
        ld = rows.shape[-1]
        q = None if "d_path" in kw else rows
        gdn.gdn_kv_append(self.dims, self.cache(), self.params, q, flat[H * D:], flat[(H + HK) * D:], ld, ld, ld,
                          None if q is None else self.q, d_status=self.status, **kw)

    def attend(self, **kw):
        gdn.gdn_attend(self.dims, self.cache(), gdn.attn_params(D ** -0.5), self.q, self.out, self.space, self.space_bytes,
                       d_status=self.status, **kw)

    def held(self, s, n):
        """Positions 0 .. n-1 of a slot as the pools hold them: k, v [n][HK][D]."""
        at = torch.arange(n, device="cuda")
        page = self.table[s].long()[at // PAGE]
        return [x.view(self.c.n_pages, HK, PAGE, D)[page, :, at % PAGE] for x in (self.k, self.v)]


def rows_of(seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, T, (H + 2 * HK) * D), generator=g).to(torch.bfloat16).cuda()


def test_tree_step_on_both_sides():
    a = Attention([37, 0, 200], seed=1)
    parent = a.c.parents()
    for s in range(B):
        parent[s, 1:] = parent[s, 1:].clamp(min=0)         # one root: the last committed token
    d_parent = parent.cuda()
    # what the target samples at each node, and drafts that follow it half of the time
    g = torch.Generator().manual_seed(2)
    tokens = torch.randint(0, 4, (B, T), generator=g, dtype=torch.int32)
    draft = torch.where(torch.rand((B, T), generator=g) < 0.6, tokens.gather(1, parent.clamp(min=0).long()),
                        torch.randint(0, 4, (B, T), generator=g, dtype=torch.int32))
    # ---- the recurrent layer's side
    dims = gdn.make_dims(B, GB["Hk"], GB["Hv"], GB["dk"], GB["dv"], T)
    C = 2 * GB["Hk"] * GB["dk"] + GB["Hv"] * GB["dv"]
    r = lambda *x, dt=torch.bfloat16: torch.randn(x, generator=g).to(dt).cuda()  # noqa: E731
    f32 = torch.float32
    weights = (r(4, C, dt=f32) * 0.5, torch.rand(GB["Hv"], generator=g).cuda(), r(GB["Hv"], dt=f32), 1 + r(GB["dv"], dt=f32) * 0.1)
    params = gdn.layer_params(*weights)
    qkv, z, alpha, beta = r(B, T, C), r(B, T, GB["Hv"] * GB["dv"]), r(B, T, GB["Hv"]), r(B, T, GB["Hv"])
    state, conv = r(B, GB["Hv"], GB["dv"], GB["dk"], dt=f32) * 0.1, r(B, 3, C, dt=f32)
    cap_state = torch.empty((B, T, GB["Hv"], GB["dv"], GB["dk"]), device="cuda")
    cap_conv = torch.empty((B, T, 3, C), device="cuda")
    out = torch.empty((B, T, GB["Hv"] * GB["dv"]), dtype=torch.bfloat16, device="cuda")
    accept, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.empty((B, T), dtype=torch.int32, device="cuda")
    rows = rows_of(3)
    # ---- one step: both layers, the acceptance, both rollbacks
    gdn.gdn_verify_tree(dims, params, qkv, z, alpha, beta, d_parent, state, conv, cap_state, cap_conv, out, a.status)
    a.append(rows, d_parent=d_parent)
    a.attend(d_parent=d_parent)
    gdn.gdn_accept_tree(dims, d_parent, draft.cuda(), tokens.cuda(), None, accept, nxt, None, path, a.status)
    gdn.gdn_rollback_tree(dims, accept, state, conv, cap_state, cap_conv, a.status)
    tree_out, tree_q = a.out.clone(), a.q.clone()
    tree_k = [a.held(s, a.c.past[s] + T) for s in range(B)]
    a.append(rows, d_path=path)
    kept = (path >= 0).sum(1).to(torch.int32)
    a.past += kept
    torch.cuda.synchronize()
    assert int(a.status.item()) == 0
    # the attention of the tree, from what its append stored
    c = a.c
    c.tree = True
    held = [(k.cpu(), v.cpu()) for k, v in tree_k]
    for s, (want, size, reach) in enumerate(attend_ref(c, tree_q.cpu(), [k for k, _ in held], [v for _, v in held], parent)):
        off = (tree_out[s].cpu().double() - want).abs() - attend_bound(c, s, want, size, reach)
        assert float(off.max()) <= 0
    # the path's nodes are a chain of the tree, both sides stand at its end
    nodes = path.cpu()
    for s in range(B):
        n = int(kept[s])
        on = [int(x) for x in nodes[s, :n]]
        assert on == sorted(on) and list(reversed(line(parent[s], on[-1]))) == on and on[-1] == int(accept[s])
        assert torch.equal(state[s], cap_state[s, on[-1]])
    # the cache is what a chain of the accepted tokens would have made of it, bit for bit
    b = Attention([37, 0, 200], seed=1)
    chain = rows.clone()
    for s in range(B):
        n = int(kept[s])
        chain[s, :n] = rows[s, nodes[s, :n].long()]
    b.append(chain, d_length=kept)
    b.past += kept
    for s in range(B):
        for x, y in zip(a.held(s, c.past[s] + int(kept[s])), b.held(s, c.past[s] + int(kept[s]))):
            assert torch.equal(x, y)
    # and the next step goes on from it
    more = rows_of(4)
    for x in (a, b):
        x.append(more)
        x.attend()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and not a.out.isnan().any()
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0


def test_chain_step_in_a_graph():
    """Append, attention, acceptance and the advance of past, captured once and replayed: as the same calls outside."""
    def step(a, rows, draft, tokens, trim, dims):
        a.append(rows)
        a.attend()
        gdn.gdn_accept(dims, draft, tokens, None, trim, None, None, a.status)
        a.past += T - trim

    g = torch.Generator().manual_seed(5)
    tokens = torch.randint(0, 3, (B, T), generator=g, dtype=torch.int32).cuda()
    draft = torch.randint(0, 3, (B, T), generator=g, dtype=torch.int32).cuda()
    draft[:, 1:6] = tokens[:, :5]
    dims = gdn.make_dims(B, 1, 1, 32, 32, T)
    outs = []
    for captured in (False, True):
        a = Attention([37, 0, 200], seed=1)
        rows, trim = rows_of(6), torch.zeros(B, dtype=torch.int32, device="cuda")
        args = (a, rows, draft, tokens, trim, dims)
        if captured:
            past = a.past.clone()
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                step(*args)
            torch.cuda.synchronize()
            a.past.copy_(past)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step(*args)
        got = []
        for i in range(2):
            rows.copy_(rows_of(7 + i))
            graph.replay() if captured else step(*args)
            torch.cuda.synchronize()
            got.append((a.out.clone(), a.past.clone()))
        assert int(a.status.item()) == 0
        outs.append(got)
    for (x, p), (y, q) in zip(*outs):
        assert torch.equal(x, y) and torch.equal(p, q)
