"""Limits of w4a16_kv4_fork: the entries of the new table are counted in 32 bits.  Host code only."""
import pytest

from test_tree_ops_abi import FORK, SHAPE, refused, w4


@pytest.mark.parametrize("rows,width", [(2048, 1 << 20), (2048, (1 << 19) + 1), (65, 1 << 24)])
def test_tables_past_the_count_are_refused(rows, width):
    """2048 rows of 2^20 entries could ask for 2^31 pages, which wrapped: nothing missing, entries unwritten."""
    assert rows * width > 1 << 30 and width * FORK["page"] <= 1 << 30
    refused(w4.w4a16_kv4_fork, SHAPE, *{**FORK, "batch_out": rows, "width": width}.values())


@pytest.mark.parametrize("rows,width", [(2048, 1 << 19), (64, 1 << 24)])
def test_tables_within_it_are_not(rows, width):
    with pytest.raises(w4.W4A16Error) as e:  # refused behind the shapes: an output that is an input
        w4.w4a16_kv4_fork(*{**FORK, "batch_out": rows, "width": width, "lens_out": FORK["lens"]}.values(), stream=0)
    assert e.value.code == -8
