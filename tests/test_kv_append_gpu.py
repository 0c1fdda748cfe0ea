"""gdn_kv_append against plain 64-bit rotations; every other place of the pools and of the output stays as it was."""
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.attn_ref import Append, Case, append_bound, line

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


class Run:
    def __init__(self, c, rope=None, norm=True, adjacent=False, path=False, base=1e6, pad=0):
        self.c, self.path = c, None
        rope = c.D if rope is None else rope
        c.pages()
        self.width = (c.H + 2 * c.Hk) * c.D
        self.ld = self.width + pad
        self.rows = c.rand(c.B, c.T, self.ld)
        self.freq = (base ** (-torch.arange(rope // 2, dtype=torch.float64) / max(1, rope // 2))).float()
        norms = [0.5 + torch.rand(c.D, generator=c.g) if norm else None for _ in range(2)]
        eps = 1e-6
        self.of_q, self.of_k = (Append(rope, self.freq, w, eps, adjacent) for w in norms)
        self.parent = c.parents() if c.tree else None
        if path:
            on = torch.rand((c.B, c.T), generator=c.g) < 0.4
            on[:, 0] = True
            self.path = torch.full((c.B, c.T), -1, dtype=torch.int32)
            for s in range(c.B):
                nodes = on[s, :c.n(s)].nonzero().flatten()
                self.path[s, :len(nodes)] = nodes
        self.kp, self.vp = c.pool(3.0), c.pool(5.0)
        self.gpu = {k: v.cuda() for k, v in dict(k=self.kp, v=self.vp, table=c.table, rows=self.rows, freq=self.freq,
                                                past=torch.tensor(c.past, dtype=torch.int32)).items()}
        self.norms = [w.cuda() if w is not None else None for w in norms]
        self.params = gdn.qk_params(rope, self.gpu["freq"] if rope else None, *self.norms, norm_eps=eps, adjacent=adjacent)
        opt = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.d = dict(d_length=torch.tensor(c.length, dtype=torch.int32).cuda() if c.length is not None else None,
                      d_parent=opt(self.parent), d_path=opt(self.path))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((c.B * c.T * c.H * c.D + 64,), 77.0, dtype=c.dtype, device="cuda")

    def call(self):
        c, g = self.c, self.gpu
        flat = g["rows"].view(-1)
        q, k, v = (flat[i * c.D:] for i in (0, c.H, c.H + c.Hk))
        has_q = self.path is None
        gdn.gdn_kv_append(c.dims(), gdn.kv_cache(g["k"], g["v"], g["table"], g["past"]), self.params, q if has_q else None,
                          k, v, self.ld, self.ld, self.ld, self.q_out if has_q else None, d_status=self.status, **self.d)

    def check(self, status=0, skip=()):
        """skip: (slot, token) whose keys and values are not written."""
        torch.cuda.synchronize()
        c = self.c
        assert int(self.status.item()) == status
        k, v, q = self.gpu["k"].cpu(), self.gpu["v"].cpu(), self.q_out.cpu()
        assert (q[c.B * c.T * c.H * c.D:] == 77).all()
        q = q[:c.B * c.T * c.H * c.D].view(c.B, c.T, c.H, c.D)
        heads = self.rows[..., :self.width].view(c.B, c.T, c.H + 2 * c.Hk, c.D)
        for s in range(c.B):
            for t in range(c.T):
                source = t if self.path is None else int(self.path[s, t])
                if t >= c.n(s) or source < 0:
                    assert (q[s, t] == 77).all()
                    continue
                depth = len(line(self.parent[s], t)) - 1 if c.tree else t
                x = heads[s, source]
                if self.path is None:
                    y, size = self.of_q(x[:c.H], c.past[s] + depth)
                    off = (q[s, t].double() - y).abs() - append_bound(c, y, size)
                    assert float(off.max()) <= 0, ("q", s, t, float(off.max()))
                if (s, t) in skip:
                    continue
                page, at = c.where(s, c.past[s] + t)
                y, size = self.of_k(x[c.H:c.H + c.Hk], c.past[s] + depth)
                off = (c.rows(k)[page, :, at].double() - y).abs() - append_bound(c, y, size)
                assert float(off.max()) <= 0, ("k", s, t, float(off.max()))
                assert torch.equal(c.rows(v)[page, :, at], x[c.H + c.Hk:])
                c.rows(k)[page, :, at] = 3.0
                c.rows(v)[page, :, at] = 5.0
        assert (k == 3).all() and (v == 5).all()


CASES = {
    "one token": (dict(T=1, H=24, Hk=4, D=256, page=16, past=[0]), dict(rope=64)),
    "one token, all rotated": (dict(T=1, H=8, Hk=2, D=128, page=64, past=[1000, 63, 64]), {}),
    "no norm": (dict(T=5, H=4, Hk=4, D=64, page=8, past=[3, 100]), dict(norm=False)),
    "no rotation": (dict(T=5, H=4, Hk=1, D=64, page=8, past=[3, 100]), dict(rope=0)),
    "neither": (dict(T=3, H=5, Hk=5, D=128, page=32, past=[30, 31]), dict(rope=0, norm=False)),
    "rope 16": (dict(T=4, H=6, Hk=2, D=128, page=16, past=[12]), dict(rope=16)),
    "rope 48": (dict(T=4, H=6, Hk=2, D=64, page=16, past=[12]), dict(rope=48)),
    "rope 240": (dict(T=2, H=6, Hk=2, D=256, page=16, past=[12]), dict(rope=240)),
    "adjacent": (dict(T=6, H=8, Hk=2, D=256, page=64, past=[500]), dict(adjacent=True)),
    "adjacent, part": (dict(T=6, H=8, Hk=2, D=64, page=64, past=[500]), dict(adjacent=True, rope=32, norm=False)),
    "far": (dict(T=3, H=4, Hk=1, D=128, page=256, past=[2 ** 20 - 5, 300001]), dict(base=10.0)),
    "ragged": (dict(T=9, H=7, Hk=7, D=128, page=8, past=[10, 0, 99, 5], length=[9, 0, 1, 6]), {}),
    "tree": (dict(T=16, H=8, Hk=2, D=128, page=16, past=[7, 1000], tree=True), {}),
    "tree of 64": (dict(T=64, H=2, Hk=1, D=64, page=32, past=[0, 33], tree=True, length=[64, 30]), {}),
    "path": (dict(T=16, H=8, Hk=2, D=128, page=16, past=[7, 1000]), dict(path=True)),
    "path of 64": (dict(T=64, H=9, Hk=3, D=64, page=8, past=[0, 91, 5], length=[64, 40, 1]), dict(path=True)),
    "padded rows, gaps": (dict(T=3, H=8, Hk=2, D=64, page=16, past=[14, 15, 16], gap=24), dict(pad=40)),
    "many tokens": (dict(T=700, H=3, Hk=1, D=64, page=64, past=[100, 5]), dict(rope=32)),
    "many heads": (dict(T=2, H=130, Hk=65, D=64, page=8, past=[6]), {}),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_cases(name, dtype):
    sizes, more = CASES[name]
    r = Run(Case(dtype=dtype, **sizes), **more)
    r.call()
    r.call()                                     # again: the same from the same
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_queries(dtype):
    c = Case(dtype=dtype, T=5, H=6, Hk=2, D=128, page=16, past=[30, 7])
    r = Run(c)
    r.call()
    torch.cuda.synchronize()
    q = r.rows[..., :c.H * c.D].contiguous().cuda()
    kv = r.gpu["rows"].view(-1)
    gdn.gdn_kv_append(c.dims(), gdn.kv_cache(r.gpu["k"], r.gpu["v"], r.gpu["table"], r.gpu["past"]), r.params, q,
                      kv[c.H * c.D:], kv[(c.H + c.Hk) * c.D:], c.H * c.D, r.ld, r.ld, q, d_status=r.status)
    torch.cuda.synchronize()
    assert torch.equal(q.view(-1), r.q_out[:q.numel()])
    r.check()


def test_bad_lengths_pages_and_nodes():
    c = Case(T=4, H=4, Hk=2, D=64, page=8, past=[20, 5, 11])
    r = Run(c)
    room = c.max_pages * c.page
    for past in (-1, room - 3, 2 ** 31 - 1):
        r.gpu["past"][1] = past
        r.status.zero_()
        r.q_out.fill_(77)
        r.gpu["k"].copy_(r.kp)
        r.gpu["v"].copy_(r.vp)
        r.call()
        keep, c.length = c.length, [4, 0, 4]
        r.check(status=gdn.GDN_ERR_LENGTH)
        c.length = keep
    r = Run(Case(T=4, H=4, Hk=2, D=64, page=8, past=[20, 5, 11]))
    r.gpu["table"][2, 1] = r.c.n_pages                # positions 8 .. 15: tokens 0 .. 3 of slot 2
    r.gpu["table"][1, 1] = -1                         # position 8: token 3 of slot 1
    r.call()
    r.check(status=gdn.GDN_ERR_PAGE, skip={(2, 0), (2, 1), (2, 2), (2, 3), (1, 3)})
    r = Run(Case(T=6, H=4, Hk=2, D=64, page=8, past=[20, 5], tree=True))
    bad = r.parent.clone()
    bad[0, 2], r.parent[0, 2] = 2, -1
    bad[1, 5], r.parent[1, 5] = -9, -1
    r.d["d_parent"] = bad.cuda()
    r.call()
    r.check(status=gdn.GDN_ERR_TREE)
    r = Run(Case(T=6, H=4, Hk=2, D=64, page=8, past=[20, 5]), path=True)
    bad = r.path.clone()
    bad[0, 0], r.path[0, 0] = 6, -1
    bad[1, 0], r.path[1, 0] = -2, -1
    r.d["d_path"] = bad.cuda()
    r.call()
    r.check(status=gdn.GDN_ERR_TREE)
