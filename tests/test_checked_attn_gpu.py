"""The test build's bounds checks on the append and the attention: no access falls outside its buffer, the results are those of
the ordinary build, bit for bit, and a buffer that the checks take for shorter than it is makes them report."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests import checked_attn_cases as cases
from tests.gpu_util import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked(tmp_path_factory):
    import __graft_entry__
    __graft_entry__.build()
    from gated_deltanet_verify_gb300 import _build
    _build.build(checked=True)
    out = tmp_path_factory.mktemp("checked") / "attn.npz"
    r = subprocess.run([sys.executable, "-m", "tests.checked_attn_cases", str(out)], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return dict(np.load(out))


def test_runs_clean_and_matches(checked):
    torch.cuda.set_device(0)
    ref = cases.run_all()
    assert "checked" not in gdn.gdn_version()
    assert set(ref) == {k for k in checked if not k.startswith("short ")}
    for k in ref:
        if k.endswith("status"):
            assert checked[k][0] == ref[k][0] == gdn.GDN_OK, k
        else:
            assert np.array_equal(ref[k], checked[k]), k


@pytest.mark.parametrize("kind,dtype,buffer", cases.SHORT)
def test_a_shorter_buffer_is_reported(checked, kind, dtype, buffer):
    assert checked[f"short {kind} {dtype} {buffer}"][0] == gdn.GDN_ERR_BOUNDS


def test_the_ordinary_build_ignores_the_switch(monkeypatch):
    torch.cuda.set_device(0)
    monkeypatch.setenv("GDN_TEST_SHORT", "past")
    for kind, sizes in (("attend", cases.SHORT_ATTEND), ("append", cases.SHORT_APPEND)):
        assert cases.call(kind, "bf16", sizes, {})[1] == gdn.GDN_OK
