"""What pda_accept_tokens refuses of its output's place.  No GPU needed."""
import ctypes

import pytest

from paged_kv_gqa_block_gb300 import _build

INVALID = -1
BASE = 1 << 20


@pytest.mark.parametrize("B,width,MB", [(3, 5, 4), (64, 1, 16)])
def test_out_lens_lie_over_no_input(B, width, MB):
    """The CTAs of a sequence read its path and table while one of them writes its length.  Addresses are never read: every call here
    is refused."""
    _build.build()
    import paged_kv_gqa_block_gb300 as pda
    p = pda.plan(B, 2, 8, 16, MB)
    at = lambda k, off=0: ctypes.c_void_p(BASE * (k + 1) + off)
    sizes = {1: 4 * B * MB, 2: 4 * B, 3: 4 * B * width, 4: 4 * B}      # table, lengths, path, its lengths
    for k, n in sizes.items():
        for out in (at(k), at(k, 4), at(k, n - 4), at(k, 4 - 4 * B)):
            rc = pda.lib().pda_accept_tokens(ctypes.byref(p), at(0), 100, at(1), at(2), at(3), at(4), width, out, None, None)
            assert rc == INVALID, (k, out.value - BASE * (k + 1))
