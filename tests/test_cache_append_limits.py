"""Limits of appending that sizes alone decide, on the CPU."""

import pytest
import torch

from test_cache_append import UNSUPPORTED, _call, lib  # noqa: F401


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("rot,Hkv,expected", [(2, 100, UNSUPPORTED), (64, 2000, UNSUPPORTED),
                                              (2, 8, -5), (64, 100, -5)])
def test_more_blocks_than_a_grid_has(lib, four, rot, Hkv, expected):  # noqa: F811
    """Tokens and heads within their own limits, but not as blocks: unsupported, not a
    failed launch (-5: no device to run on). Inputs are the same for all tokens, so
    that they have room."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: nothing may launch")
    same = (0, 0, 0)
    assert _call(lib, four, q=None, qo=None, B=1, Hq=0, Hkv=Hkv, N=(1 << 31) - 256, rot=rot,
                 ks=same, vs=same, new=None, pos=None) == expected
