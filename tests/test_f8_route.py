"""Where the 8-bit floating-point products of few rows run."""

from test_group_planner import plans, pytestmark  # noqa: F401


def test_row_tiles_of_a_group_share_an_xcd(plans):  # noqa: F811
    """Neighbouring units are the row tiles of one strip: an XCD's share of them is contiguous. A plain product has one."""
    asked = [("decode", rows, groups, 0, 4096, 4096, False, False, False, 256) for rows, groups in ((64, 8), (128, 8), (64, 64), (1000, 300), (40, 0), (1, 0))]
    for a, got in zip(asked, plans(asked)):
        assert got["plan"]["nxcd"] == (8 if a[2] else 1), a
