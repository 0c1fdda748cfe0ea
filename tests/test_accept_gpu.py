"""gdn_accept and gdn_accept_tree against plain loops, and the rollbacks they feed."""
import numpy as np
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.step_ref import accept_row, accept_tree_row

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def dims_of(B, T):
    return gdn.make_dims(B, 1, 1, 32, 32, T)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def outputs(B, T, n):
    return [torch.full((B + 8,) if i < 2 else (B * T + 8,), 99, dtype=torch.int32, device="cuda") for i in range(n)]


def take(t, B, T=None):
    v = t.cpu().numpy()
    n = B if T is None else B * T
    assert (v[n:] == 99).all()
    return v[:n] if T is None else v[:n].reshape(B, T)


def draw_chain(rng, B, T):
    tokens = rng.integers(0, 6, (B, T)).astype(np.int32)
    draft = np.concatenate([rng.integers(0, 6, (B, 1)), np.where(rng.random((B, T - 1)) < 0.85, tokens[:, :-1],
                                                                 rng.integers(0, 6, (B, T - 1)))], 1).astype(np.int32)
    return draft, tokens


@pytest.mark.parametrize("T", [1, 2, 3, 16, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("B", [1, 5, 130])
def test_chain(B, T):
    rng = np.random.default_rng(B * 100 + T)
    draft, tokens = draw_chain(rng, B, T)
    draft[0, 1:] = tokens[0, :-1]                       # everything accepted
    if B > 1:
        tokens[1, : (T + 1) // 2] = -1                  # an unsampled place matches nothing, not even a draft of -1
        draft[1] = -1
    for length in (None, rng.integers(1, T + 1, B).astype(np.int32)):
        trim, nxt, emit = outputs(B, T, 3)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_accept(dims_of(B, T), up(draft), up(tokens), None if length is None else up(length), trim, nxt, emit, status)
        ref = [accept_row(draft[s].tolist(), tokens[s].tolist(), T if length is None else int(length[s]), T) for s in range(B)]
        assert take(trim, B).tolist() == [r[0] for r in ref]
        assert take(nxt, B).tolist() == [r[1] for r in ref]
        assert take(emit, B, T).tolist() == [r[2] for r in ref]
        assert int(status) == 0


def draw_tree(rng, B, T):
    parent = np.full((B, T), -1, dtype=np.int32)
    for t in range(1, T):
        parent[:, t] = np.maximum(0, t - 1 - (rng.random(B) ** 2 * min(t, 6)).astype(np.int32))
    tokens = rng.integers(0, 3, (B, T)).astype(np.int32)
    draft = rng.integers(0, 3, (B, T)).astype(np.int32)   # few values: twins among a node's children
    return parent, draft, tokens


@pytest.mark.parametrize("T", [1, 2, 5, 16, 32, 33, 64])
@pytest.mark.parametrize("B", [1, 7, 129])
def test_tree(B, T):
    rng = np.random.default_rng(B * 1000 + T)
    parent, draft, tokens = draw_tree(rng, B, T)
    if T > 1:
        parent[0, T // 2] = -1                          # a second root is no error and never reached
    parent[-1] = np.arange(T) - 1                       # a chain that agrees all along
    draft[-1, 1:] = tokens[-1, :-1]
    for length in (None, rng.integers(0, T + 1, B).astype(np.int32)):
        acc, nxt, emit, path = outputs(B, T, 4)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        gdn.gdn_accept_tree(dims_of(B, T), up(parent), up(draft), up(tokens), None if length is None else up(length), acc,
                            nxt, emit, path, status)
        ref = [accept_tree_row(parent[s].tolist(), draft[s].tolist(), tokens[s].tolist(),
                               T if length is None else int(length[s]), T) for s in range(B)]
        for got, i, wide in ((acc, 0, None), (nxt, 1, None), (emit, 2, T), (path, 3, T)):
            assert take(got, B, wide).tolist() == [r[i] for r in ref]
        assert int(status) == 0


def test_the_optional_outputs_may_be_left_out():
    rng = np.random.default_rng(0)
    draft, tokens = draw_chain(rng, 3, 6)
    trim, = outputs(3, 6, 1)
    gdn.gdn_accept(dims_of(3, 6), up(draft), up(tokens), None, trim)
    assert take(trim, 3).tolist() == [accept_row(draft[s].tolist(), tokens[s].tolist(), 6, 6)[0] for s in range(3)]
    parent, draft, tokens = draw_tree(rng, 3, 6)
    acc, = outputs(3, 6, 1)
    gdn.gdn_accept_tree(dims_of(3, 6), up(parent), up(draft), up(tokens), None, acc)
    assert take(acc, 3).tolist() == [accept_tree_row(parent[s].tolist(), draft[s].tolist(), tokens[s].tolist(), 6, 6)[0]
                                     for s in range(3)]


@pytest.mark.parametrize("bad", [0, -1, 7])
def test_a_bad_length_keeps_nothing_of_its_slot(bad):
    rng = np.random.default_rng(1)
    T, B = 6, 3
    draft, tokens = draw_chain(rng, B, T)
    length = np.array([T, bad, 2], dtype=np.int32)
    trim, nxt, emit = outputs(B, T, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_accept(dims_of(B, T), up(draft), up(tokens), up(length), trim, nxt, emit, status)
    ref = [accept_row(draft[s].tolist(), tokens[s].tolist(), int(length[s]), T) for s in range(B)]
    assert take(trim, B).tolist() == [r[0] for r in ref] and take(trim, B)[1] == -1 and take(nxt, B)[1] == -1
    assert (take(emit, B, T)[1] == -1).all() and int(status) == gdn.GDN_ERR_LENGTH
    parent, draft, tokens = draw_tree(rng, B, T)
    acc, nxt, emit, path = outputs(B, T, 4)
    status.zero_()
    gdn.gdn_accept_tree(dims_of(B, T), up(parent), up(draft), up(tokens), up(length), acc, nxt, emit, path, status)
    assert take(acc, B)[1] == -1 and (take(path, B, T)[1] == -1).all()
    assert int(status) == (0 if bad == 0 else gdn.GDN_ERR_LENGTH)      # a tree slot may be empty


@pytest.mark.parametrize("t,p", [(0, 0), (0, -2), (2, 2), (2, 5), (3, -2)])
def test_a_bad_parent_is_reported_and_not_reached(t, p):
    T = 5
    parent = np.array([[-1, 0, 1, 2, 3]] * 2, dtype=np.int32)
    tokens = np.full((2, T), 4, dtype=np.int32)
    draft = np.full((2, T), 4, dtype=np.int32)
    parent[1, t] = p
    acc, nxt, emit, path = outputs(2, T, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_accept_tree(dims_of(2, T), up(parent), up(draft), up(tokens), None, acc, nxt, emit, path, status)
    assert take(acc, 2).tolist() == [4, t - 1] and int(status) == gdn.GDN_ERR_TREE
    assert take(path, 2, T)[1].tolist() == list(range(t)) + [-1] * (T - t)
