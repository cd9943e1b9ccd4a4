"""Host-only refusals of the cache's upkeep: outputs that lie over inputs."""
from __future__ import annotations

import pytest

from paged_fp8_speculative_gb300 import api
from tests.test_tree_host import COMPACT, COMPACT_GOOD, FAKE, RESIZE, RESIZE_GOOD, call

FAR = FAKE + (1 << 20)


@pytest.mark.parametrize("name,words", [("sl", 2), ("count", 2), ("cu", 3), ("index", 2 * 8), ("bt", 2 * 4)])
def test_compact_refuses_new_lengths_over_an_input(name, words):
    """Two sequences, paths 8 wide, tables 4 wide; the new lengths on any word of an input, and one
    word before and behind it."""
    for first in range(-2, words + 2):
        over = {name: FAR, "new": FAR + 4 * first}
        rc = call("mtp_cache_compact", COMPACT, COMPACT_GOOD, **over)
        if -2 < first < words:
            assert rc == api.E_ARG, first
        else:                                       # nothing but the pointers themselves is wrong
            assert rc == api.E_DEVICE, first


def test_resize_refuses_new_lengths_over_the_lengths():
    for first in range(-3, 5):                      # three rows
        rc = call("mtp_cache_resize", RESIZE, RESIZE_GOOD, sl=FAR, new=FAR + 4 * first)
        assert rc == (api.E_ARG if -3 < first < 3 else api.E_DEVICE), first
