"""examples/losses_of_logits.py runs, and each of its stages learns."""
import importlib.util
import os

import pytest

from conftest import ROOT
from gpu_util import lib_ready

pytestmark = pytest.mark.gpu


def test_every_stage_learns():
    lib_ready()
    path = os.path.join(ROOT, "examples", "losses_of_logits.py")
    spec = importlib.util.spec_from_file_location("losses_of_logits", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    d, p, r, v = example.main()
    assert d[-1] < 0.5 * d[0]
    assert p[-1][0] < 0.5 * p[0][0] and p[-1][2] > 0.9
    assert r[-1] > r[0] + 0.1
    assert v[-1] > v[0] + 0.3
