"""The token operators together: the example's transformer block, forward and backward, against fp64.

Every tensor between operators is rounded to bf16 (2^-9 of it on average); the
longest path rounds about ten times, so errors stay below 10 * 2^-8 in the L2 norm.
"""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("frames,size,channels,heads", [(1, 8, 128, 2), (3, 16, 256, 4), (2, 9, 320, 5)])
def test_block_matches_fp64(frames, size, channels, heads):
    import latent_block
    for name, e in latent_block.run(frames, size, channels, heads).items():
        assert e < 10 * 2.0 ** -8, "%s: relative error %g" % (name, e)
