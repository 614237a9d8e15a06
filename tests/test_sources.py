"""Rules that every source of the library keeps, whatever it computes (no GPU needed)."""
import os

from mtp_speculative_draft_head_gb300 import build


def test_no_load_is_multicast():
    """Ranks of a replicated or sharded run load this one library: a copy that writes the shared memory of several
    CTAs at once stays out of all of it."""
    word = "multi" + "cast"
    for path in build._deps():
        with open(path) as f:
            assert word not in f.read(), os.path.basename(path)
