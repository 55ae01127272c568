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


def test_read_only_loads():
    """Kernels that start while the kernel before them still runs may not read
    through the read-only path what that kernel writes.  The decode attention
    starts when the call's first kernel has waited for everything before it and
    reads the context lengths, which its own call does not write, that way;
    no other latent kernel uses it."""
    for p in SOURCES:
        if p.name.startswith("latent_"):
            lines = [x for x in p.read_text().splitlines() if re.search(r"__ldg\b|ld\.global\.nc", x)]
            if p.name == "latent_decode.cu":
                lines = [x for x in lines if "__ldg(a.ctx_lens + b)" not in x]
            assert not lines, (p.name, lines)
