"""The example trains: its loss falls from about log(vocabulary) towards what the data's noise leaves."""
import importlib.util
import math
import os

import pytest

from tests.helpers import ROOT


@pytest.mark.gpu
def test_clipped_training_learns():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("clipped_training", os.path.join(ROOT, "examples", "clipped_training.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, clipped = ex.train(steps=60, ranks=4, log=lambda *a: None)
    assert all(math.isfinite(x) for x in losses)
    assert losses[0] > 4.0           # near log(500) = 6.2 before training, less or more by the random head
    assert losses[-1] < losses[0] / 2
    assert clipped > 0
