"""Static checks on the attention kernels' sources (CPU): roles wait as whole warps, and every wait has a deadline."""
import re

from test_wait_rules import code


def test_roles_wait_as_whole_warps():
    text = code("attend_many.cuh")
    assert "mbar_wait_warp(" in text and not re.search(r"\bmbar_wait\(", text)


def test_register_split_fits_the_launch():
    """setmaxnreg shares of the four warpgroups against the 128 registers a thread that the launch has."""
    text = code("attend_many.cuh")
    shares = [int(x) for x in re.findall(r"setmaxnreg\.(?:inc|dec)\.sync\.aligned\.u32 (\d+);", text)]
    threads = int(re.search(r"kAmThreads = (\d+);", text).group(1))
    assert threads == 512 and len(shares) == 3                 # converters, products and copies, softmax (two warpgroups)
    assert 128 * (shares[0] + shares[1] + 2 * shares[2]) <= threads * 128
    assert all(x % 8 == 0 and 24 <= x <= 256 for x in shares)
