"""Appends and attentions run through both the ordinary and the bounds-checked library (see test_checked_attn_gpu.py).
``python -m tests.checked_attn_cases OUT.npz`` runs them on the checked library and saves the results and status words."""
import os
import sys

import numpy as np
import torch

import gated_deltanet_verify_gb300 as gdn
from tests import test_attend_gpu as attend
from tests import test_kv_append_gpu as append
from tests.attn_ref import Case

ATTEND = {
    "one token": dict(T=1, H=8, Hk=2, D=128, page=16, past=[126, 127, 128, 129, 3000]),
    "ragged": dict(T=7, H=12, Hk=4, D=256, page=32, past=[300, 0, 40, 999, 12, 0], length=[7, 1, 0, 3, 6, 0]),
    "rows of 8": dict(T=2, H=8, Hk=2, D=64, page=16, past=[5000, 61]),
    "rows of 16": dict(T=5, H=6, Hk=2, D=128, page=16, past=[2500, 0, 61], length=[5, 5, 3]),
    "rows of 32": dict(T=9, H=6, Hk=2, D=256, page=8, past=[1500, 61]),
    "chunk": dict(T=150, H=8, Hk=2, D=128, page=64, past=[130, 5, 600], length=[150, 1, 97]),
    "tree": dict(T=64, H=8, Hk=2, D=64, page=32, past=[120, 0, 1000], tree=True, length=[64, 33, 2]),
    "window, sinks": dict(T=5, H=8, Hk=2, D=128, page=16, past=[2000, 130, 3, 700], window=64, n_sink=4, gap=8 * 13),
    "window over tree": dict(T=40, H=6, Hk=2, D=256, page=256, past=[0, 200, 1000], window=7, n_sink=3, tree=True),
    "more slots than a warp looks through": dict(T=1, H=4, Hk=2, D=128, page=8, past=[(91 * i) % 300 for i in range(300)]),
    "more blocks than a warp looks through": dict(T=1100, H=32, Hk=1, D=64, page=64, past=[40]),
}
APPEND = {
    "one token": (dict(T=1, H=24, Hk=4, D=256, page=16, past=[0]), dict(rope=64)),
    "ragged": (dict(T=9, H=7, Hk=7, D=128, page=8, past=[10, 0, 99, 5], length=[9, 0, 1, 6]), {}),
    "adjacent, padded rows, gaps": (dict(T=3, H=8, Hk=2, D=64, page=16, past=[14, 15, 16], gap=24), dict(pad=40, adjacent=True)),
    "tree": (dict(T=64, H=2, Hk=1, D=64, page=32, past=[0, 33], tree=True, length=[64, 30]), {}),
    "path": (dict(T=64, H=9, Hk=3, D=64, page=8, past=[0, 91, 5], length=[64, 40, 1]), dict(path=True)),
    "many tokens": (dict(T=700, H=3, Hk=1, D=128, page=64, past=[100, 5]), dict(rope=32, norm=False)),
}
# with one buffer taken for half as long as it is
SHORT_ATTEND = dict(T=2, H=8, Hk=2, D=128, page=16, past=[3000, 2900, 2000, 2990])
SHORT_APPEND = dict(T=6, H=8, Hk=2, D=128, page=16, past=[30, 29, 20, 28])


def call(kind, dtype, sizes, more):
    c = Case(dtype=dtype, **sizes)
    r = attend.Run(c) if kind == "attend" else append.Run(c, **more)
    r.call()
    torch.cuda.synchronize()
    out = dict(out=r.out) if kind == "attend" else dict(q=r.q_out, k=r.gpu["k"], v=r.gpu["v"])
    return {n: x.contiguous().view(torch.uint8).cpu().numpy() for n, x in out.items()}, int(r.status.item())


def run_all() -> dict:
    torch.cuda.set_device(0)
    res = {}
    for dtype in ("f32", "bf16"):
        for kind, cases in (("attend", {k: (v, {}) for k, v in ATTEND.items()}), ("append", APPEND)):
            for name, (sizes, more) in cases.items():
                out, status = call(kind, dtype, sizes, more)
                key = f"{kind} {dtype} {name}"
                res[key + " status"] = np.array([status])
                res.update({f"{key} {n}": x for n, x in out.items()})
    return res


SHORT = ([("attend", d, b) for d in ("f32", "bf16") for b in ("past", "table", "nodes", "q", "partial", "stats")] +
         [("attend", "f32", "pool")] +           # (in bf16 pages come as boxes, which end with the tensor)
         [("append", d, b) for d in ("f32", "bf16") for b in ("past", "table", "nodes", "path", "q", "k", "v", "out", "freq", "norm", "pool")])


def run_short() -> dict:
    res = {}
    for kind, dtype, buffer in SHORT:
        os.environ["GDN_TEST_SHORT"] = "nodes" if buffer == "path" else buffer
        sizes = dict(SHORT_ATTEND if kind == "attend" else SHORT_APPEND, tree=buffer == "nodes")
        _, status = call(kind, dtype, sizes, dict(path=buffer == "path"))
        del os.environ["GDN_TEST_SHORT"]
        res[f"short {kind} {dtype} {buffer}"] = np.array([status])
    return res


if __name__ == "__main__":
    from gated_deltanet_verify_gb300 import _build
    gdn.LIB_PATH = _build.CHECKED_LIB
    r = run_all()
    r.update(run_short())
    assert "checked" in gdn.gdn_version()
    np.savez(sys.argv[1], **r)
