"""The attention's workspace, held against the tiles that a call's rows make."""
import pytest

from test_serving_abi import att, kv, q, refused  # noqa: F401  (q is the fixture)

WORKGROUPS = 512  # that a split call is cut for


def tile_rows(B, n, group, heads, length):
    """Rows of a tile: sixteen while rows are few or their tiles and pages are, else 64 where tiles of 128 are few and
    sequences short, else 128."""
    rows, pages = n * group, -(-length // 64)
    sixteens = -(-rows // 16) * B * heads
    few = rows <= 48 or sixteens <= 512 if pages <= 16 else rows <= 96 or sixteens <= 16384 // pages
    if few:
        return 16
    return 64 if -(-rows // 128) * B * heads < 256 and pages <= 48 else 128


@pytest.mark.parametrize("D,heads,group", [(128, 8, 4), (64, 1, 1), (64, 2, 7), (256, 4, 2), (128, 32, 1)])
def test_one_part_a_tile_and_those_that_fill_the_device(q, D, heads, group):
    """A split call has one part a tile and at most WORKGROUPS more over all heads (or as many as chunks of eight pages
    make, if these are fewer); one that is not has none."""
    split = 0
    for B in (1, 2, 5, 64, 200, 256, 257, 1000):
        for n in (1, 3, 9, 24, 25, 33, 70, 700):
            c = kv(q, heads=heads, dim=D)
            for length in (n, 400, 1500, 2000, 4000, 10000, 1 << 20):
                length = max(n, length)
                need = q.qattend_workspace_bytes(c, heads * group, B, B * n, n, length)
                rows = tile_rows(B, n, group, heads, length)
                tiles, pages = B * -(-n * group // rows), -(-length // 64)
                items = min(tiles + -(-WORKGROUPS // heads), tiles * (1 + pages // 8))
                parts = items * heads * rows
                assert need in (0, -(-parts * D * 4 // 256) * 256 + parts * 8), (B, n, length, rows)
                if pages > 32 and B <= 256 and tiles * heads < WORKGROUPS:
                    assert need > 0
                if pages <= 24 or B > 256 or tiles * heads >= 4 * WORKGROUPS:
                    assert need == 0
                split += need > 0
    assert split > 40


def test_smaller_limits_may_need_more(q):
    """A workspace of one shape's size does not serve every smaller one: it is refused, not overrun."""
    c = kv(q, heads=8, dim=128, pages=1000)
    large, small = [q.qattend_workspace_bytes(c, 32, B, 5 * B, 5, 10000) for B in (300, 64)]
    assert large == 0 < small
    refused(q, "Q8K_ERR_WORKSPACE", lambda: att(q, cache=c, heads=32, qs=4096, B=64, Tq=320, max_q=5, max_pages=200,
                                                max_len=10000, ws=None, wsb=large))
