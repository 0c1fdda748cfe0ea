"""One verify step decided on the device: the layer with adapters, sampling, acceptance and the rollback, chained on
one stream and as a CUDA graph, against the same step decided on the host."""
import numpy as np
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.gpu_util import dims_of, params_of, upload
from tests.step_ref import accept_row, accept_tree_row, sample_row
from tests.test_lora_gpu import Case, shape_of
from workloads.device import empty_outputs
from workloads.synth import make_inputs, make_parents

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


V = 41                      # a small vocabulary, so that drafts agree now and then


class Step:
    def __init__(self, seed, tree=False):
        s = self.shape = shape_of(n_slots=6, n_tokens=7, n_embd=128)
        B, T = s.n_slots, s.n_tokens
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = [0, -1, 1, 2, 2, 0]
        self.i, self.o = Case(s, "in", 3, 16, ids, seed=seed), Case(s, "out", 3, 8, ids, seed=seed + 1)
        self.tree = tree
        self.inp = make_inputs(s)
        self.parent = torch.from_numpy(make_parents(s).astype(np.int32)).cuda()
        if tree:
            self.parent[:, 0] = -1
            self.parent[:, 1:].clamp_(min=0)
        self.head = torch.randn((s.n_embd, V), generator=g, device="cuda")
        self.draft = torch.randint(0, 4, (B, T), generator=g, device="cuda", dtype=torch.int32)
        self.u = torch.rand((B, T), generator=g, device="cuda")
        self.params = (torch.tensor([0.0, 1.0, 0.7, 1.2, 0.0, 0.9], device="cuda"),
                       torch.tensor([0, 4, 0, 0, 3, 6], dtype=torch.int32, device="cuda"),
                       torch.tensor([1.0, 1.0, 0.8, 1.0, 1.0, 0.9], device="cuda"),
                       torch.tensor([0.0, 0.0, 0.0, 0.1, 0.0, 0.05], device="cuda"))
        i32 = lambda *sh: torch.empty(sh, dtype=torch.int32, device="cuda")  # noqa: E731
        self.tokens, self.place, self.next, self.emit, self.path = i32(B, T), i32(B), i32(B), i32(B, T), i32(B, T)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dims = dims_of(s)
        self.size = gdn.gdn_layer_lora_workspace_bytes(self.dims, s.n_embd, 16)
        self.ws = torch.empty(self.size, dtype=torch.uint8, device="cuda")
        self.y = torch.empty((B * T, s.n_embd), dtype=torch.bfloat16, device="cuda")
        self.x, self.e = upload(self.inp), empty_outputs(s, "cuda")
        self.logits = torch.empty((B * T, V), device="cuda")
        if tree:
            self.e["cap_conv"] = torch.empty((B, T, 3, s.conv_channels), device="cuda")

    def enqueue(self):
        s, x, e = self.shape, self.x, self.e
        w = gdn.proj_weights(s.n_embd, self.i.w, self.o.w)
        if not self.tree:
            gdn.gdn_layer_verify_lora(self.dims, params_of(x), w, self.i.lora, self.o.lora, self.i.ids, self.i.x, x["state"],
                                      x["conv_state"], e["cap_state"], e["cap_conv"], self.y, self.ws, self.size, self.status)
        else:
            gdn.gdn_verify_tree(self.dims, params_of(x), x["qkv"], x["z"], x["alpha"], x["beta_raw"], self.parent,
                                x["state"], x["conv_state"], e["cap_state"], e["cap_conv"], e["out"], self.status)
            gdn.gdn_project_out_lora(self.dims, w, self.o.lora, self.o.ids, e["out"], self.y, self.ws, self.size, self.status)
        torch.matmul(self.y.float(), self.head, out=self.logits)      # the model's head, here a small product
        gdn.gdn_sample(gdn.make_sample_dims(s.n_slots, s.n_tokens, V), gdn.sample_params(*self.params), self.logits, self.u,
                       self.tokens, None, self.status)
        if not self.tree:
            gdn.gdn_accept(self.dims, self.draft, self.tokens, None, self.place, self.next, self.emit, self.status)
            gdn.gdn_rollback(self.dims, self.place, x["state"], x["conv_state"], e["cap_state"], e["cap_conv"], self.status)
        else:
            gdn.gdn_accept_tree(self.dims, self.parent, self.draft, self.tokens, None, self.place, self.next, self.emit,
                                self.path, self.status)
            gdn.gdn_rollback_tree(self.dims, self.place, x["state"], x["conv_state"], e["cap_state"], e["cap_conv"],
                                  self.status)

    def guess(self):
        """Drafts that mostly agree with what was sampled (the logits do not depend on them here)."""
        T = self.shape.n_tokens
        par = self.parent.long().clamp(min=0) if self.tree else (torch.arange(T, device="cuda") - 1).clamp(min=0).expand(6, T)
        keep = torch.rand(self.draft.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)) < 0.8
        self.draft = torch.where(keep, self.tokens.gather(1, par), self.draft).contiguous()

    def restore(self):
        fresh = upload(self.inp)
        self.x["state"].copy_(fresh["state"])
        self.x["conv_state"].copy_(fresh["conv_state"])

    def check(self):
        s = self.shape
        B, T = s.n_slots, s.n_tokens
        torch.cuda.synchronize()
        assert int(self.status) == 0
        l, u = self.logits.double().cpu().numpy(), self.u.double().cpu().numpy().reshape(-1)
        par = [p.double().cpu().numpy() for p in self.params]
        tok = [sample_row(l[i], par[0][i // T], int(par[1][i // T]), par[2][i // T], par[3][i // T], u[i])[0]
               for i in range(B * T)]
        assert self.tokens.cpu().numpy().reshape(-1).tolist() == tok
        tok = np.array(tok).reshape(B, T)
        draft, parent = self.draft.cpu().numpy(), self.parent.cpu().numpy()
        kept = 0
        for b in range(B):
            if self.tree:
                place, nxt, emit, path = accept_tree_row(parent[b].tolist(), draft[b].tolist(), tok[b].tolist(), T, T)
                assert self.path[b].tolist() == path
                node = place
            else:
                place, nxt, emit = accept_row(draft[b].tolist(), tok[b].tolist(), T, T)
                node = T - 1 - place
            assert (int(self.place[b]), int(self.next[b]), self.emit[b].tolist()) == (place, nxt, emit)
            assert torch.equal(self.x["state"][b], self.e["cap_state"][b, node])
            kept += len([v for v in emit if v >= 0])
        assert B < kept < B * T            # some guesses were accepted, some were not


@pytest.mark.parametrize("tree", [False, True])
def test_a_step_on_the_device(tree):
    st = Step(7, tree)
    st.enqueue()
    torch.cuda.synchronize()
    st.guess()
    st.restore()
    st.enqueue()
    st.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):          # warm-up of the library product outside the capture
        torch.matmul(st.y.float(), st.head, out=st.logits)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.enqueue()
    for k in range(2):
        st.u.copy_(torch.rand(st.u.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(50 + k)))
        st.restore()
        st.tokens.fill_(-5)
        g.replay()
        st.check()
