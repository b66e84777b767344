"""What the paged cache's kernels may not do, seen in their sources."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sequence_long_context_zigzag_gb300", "csrc")


def test_kernels_that_start_early_do_not_use_the_read_only_path():
    """These kernels may begin before the grid that writes their inputs has ended, so their inputs are not read-only for
    their whole life."""
    files = [f for f in glob.glob(os.path.join(CSRC, "paged*.cu*"))]
    assert len(files) >= 7
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        assert not re.search(r"__ldg|\.nc\b|__restrict__", code), os.path.basename(f)
