"""What holds of the kernels' sources as text (no GPU needed)."""
import glob
import os
import re

from tests.conftest import ROOT


def sources():
    paths = sorted(glob.glob(os.path.join(ROOT, "sharded_state_gb300", "csrc", "*")))
    assert len(paths) >= 15
    return {os.path.basename(p): open(p).read() for p in paths}


def test_no_load_is_multicast():
    """Every CTA fetches its own tiles: the library also runs in processes that have several GPUs, its tensor maps are of
    whatever address a caller gives, and a multicast load is only sound within one GPU's own memory.  (The commit of a
    pair's products arrives at both CTAs' barriers, which is no load.)"""
    for name, text in sources().items():
        code = re.sub(r'"\s*"', "", text)  # neighbouring string literals are one
        for literal in re.findall(r'"([^"]*)"', code):
            if "multicast" in literal:
                assert "cp.async.bulk" not in literal and "tcgen05.commit" in literal, (name, literal)
