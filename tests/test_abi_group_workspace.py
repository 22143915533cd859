"""Grouping's workspace holds the counts of the chunks that there can be: 1024 rows each, and no more than 512."""
import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import block_scaled_mlp_gb300 as mx
    return mx.lib()


@pytest.mark.parametrize("R,E,chunks", [(8193, 64, 9), (131072, 64, 128), (512 * 1024, 256, 512), (512 * 1024 + 1, 256, 512),
                                        (1 << 24, 1024, 512), ((1 << 31) - 2048, 1, 512)])
def test_many_rows_need_no_more_than_the_chunks(L, R, E, chunks):
    assert L.mx_token_group_workspace(R, E) == chunks * E * 4
