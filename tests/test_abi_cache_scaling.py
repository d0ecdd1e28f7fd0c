"""What rope_frequencies() and rope_table() refuse of a scaling: all with the binding's own error, none with Python's (no GPU needed)."""
import math

import pytest

from mxfp8_block_scaled_07_b200 import mx

BAD = [("yarn",), ("yarn", 4), ("yarn", 4, 0), ("yarn", 4, -8), ("yarn", 4, 4096, 0), ("yarn", 4, 4096, 32, 0), ("yarn", 0, 4096),
       ("yarn", math.inf, 4096), ("yarn", math.nan, 4096), ("yarn", "4", "many"), ("ntk",), ("ntk", 0), ("ntk", -2), ("ntk", math.inf),
       ("ntk", 1e300), ("linear",), ("linear", -1), ("linear", math.nan), ("linear", None), ("cubic", 2), "yarn", 7, ([], 2), (2, 2)]


@pytest.mark.parametrize("scaling", BAD, ids=str)
def test_refusals(scaling):
    for rot in (8, 4):
        with pytest.raises(mx.MxError):
            mx.rope_frequencies(rot, 1e300, scaling)
    with pytest.raises(mx.MxError):
        mx.rope_table(4, 8, 1e300, scaling)


def test_bases():
    for base in (0, -1.0, math.nan):
        with pytest.raises(mx.MxError):
            mx.rope_frequencies(8, base)
    for base, scaling in ((1, ("yarn", 4, 4096)), (1.0, ("yarn", 4, 4096)), (5e-324, None)):
        with pytest.raises(mx.MxError):
            mx.rope_frequencies(64, base, scaling)
    assert mx.rope_frequencies(8, 1) == ([1.0] * 4, 1.0)


def test_what_is_taken():
    plain = mx.rope_frequencies(64, 1e4)
    assert mx.rope_frequencies(64, 1e4, ()) == plain == mx.rope_frequencies(64, 1e4, ("linear", 1)) == mx.rope_frequencies(64, 1e4, ["ntk", 1])
    full = mx.rope_frequencies(64, 1e4, ("yarn", 4, 4096, 32, 1))
    assert mx.rope_frequencies(64, 1e4, ("yarn", 4, 4096, 32)) == full == mx.rope_frequencies(64, 1e4, ("yarn", 4.0, 4096))
    assert mx.rope_frequencies(64, 1e4, ("yarn", 0.5, 4096))[1] == 1.0
