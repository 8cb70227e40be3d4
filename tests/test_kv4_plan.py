"""The host's choice of attention kernels, as the workspace size shows it (no GPU)."""
import pytest

import int4_group_wise_b200 as q4


@pytest.mark.parametrize("heads", [1, 2, 8, 64])
@pytest.mark.parametrize("dim", [64, 128])
def test_tall_tiles_never_come_in_clusters(heads, dim):
    """17 to 24 rows for each of 64 or more (request, kv head) pairs take tiles of 24 rows, which the one-launch form is
    not built for: such a call has a workspace, however short its table."""
    for batch in (-(-64 // heads), -(-64 // heads) + 1, 200, 65536):
        for group, new in ((4, 5), (4, 6), (17, 1), (24, 1), (1, 20)):
            n = batch * new
            if n * heads * group > 2 ** 31 - 1:
                continue
            for blocks in (1, 4, 256):
                assert q4.kv4_attention_workspace_bytes(n, batch, heads * group, heads, dim, 16, blocks) > 0
    # and the one-launch form, without a workspace, is there for small batches of lower tiles
    assert q4.kv4_attention_workspace_bytes(1, 1, 4, 1, dim, 16, 256) == 0
    assert q4.kv4_attention_workspace_bytes(20, 1, 1, 1, dim, 16, 256) == 0


def test_prompts_over_long_tables_have_a_piece_for_every_row():
    """A request of more than 2^15 tokens has its sums joined in the workspace: room for a row's output, maximum and sum
    for each head, from the first table that can name that many; without it, none where one launch does."""
    n, heads, dim = 20000, 32, 128
    row = n * heads * (dim + 2) * 4
    for page in (16, 128):
        short, long = (q4.kv4_attention_workspace_bytes(n, 1, heads, 8, dim, page, (1 << 15) // page + more) for more in (0, 1))
        assert short == 0 and row <= long < row + 256
