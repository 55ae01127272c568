"""Rules that the latent-cache kernels' sources keep (CPU)."""
import re

from decode_step_gb300.build import CSRC

SOURCES = sorted(p for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh", ".cpp", ".h"))


def test_no_copies_into_other_ctas():
    """Loads that land in several CTAs of a cluster are for programs on one GPU
    only; this library also runs as replicas on several."""
    name = re.compile("multicast" + "::")
    assert SOURCES
    for p in SOURCES:
        assert not name.search(p.read_text()), p.name
