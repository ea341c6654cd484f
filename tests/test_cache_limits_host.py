"""Sizes at the edge of what lean_prefix_attention counts in 32 bits are refused, no GPU needed."""
import pytest

from test_cache_host import cache_structs, lean, refused  # noqa: F401  (lean: the fixture)
from test_step_host import P


@pytest.mark.parametrize("page", [16, 1, 100])
def test_long_prefixes(lean, page):  # noqa: F811
    n = 300
    good = dict(n_seqs=n, n_q_heads=1, n_kv_heads=1, head_dim=64, cache_dtype=1, q=P, q_stride=64, q_head_stride=64, k_cache=P,
                v_cache=P, n_pages=4, page_size=page, page_stride=6400, place_stride=64, cache_head_stride=64, n_prefixes=1,
                prefix_table=P, prefix_width=3, prefix_stride=1 << 31, prefix_lens=P, seq_starts=P, block_table=P,
                table_width=2, table_stride=1 << 31, seq_lens=P, out=P, out_stride=64, out_head_stride=64, scale=0.125,
                workspace=P, workspace_bytes=lean.lean_prefix_attention_workspace_bytes(n, 1, 1, 64, n))
    call, fields = (lean, "lean_prefix_attention", lean._PREFIX), cache_structs()["lean_prefix_args"]
    most = (2 ** 31 - 129) // page
    tiles = most * page // 128 + 5  # of a prefix as it is counted, an item's beginning included
    refused(*call, fields, good, [
        ("SHAPE", dict(prefix_width=most + 1)),       # a tile's end would pass 2^31
        ("ALIGN", dict(prefix_width=most, q=P + 8)),  # this many are taken
        ("SHAPE", dict(prefix_width=most, n_prefixes=2 ** 32 // tiles + 1)),  # all prefixes' tiles
        ("SHAPE", dict(table_width=(2 ** 31 - 1) // page, q=P))])             # all sequences' own units
