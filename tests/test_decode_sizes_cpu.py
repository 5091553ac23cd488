"""Sizes beyond the cached attention's row numbers are refused on the host: nothing here reaches a GPU."""
from tensor_matmul_collective_gb300 import coc

from test_decode_ops_cpu import L, _desc, attend  # noqa: F401  (L: fixture)


def test_attention_refuses_more_rows_than_it_can_number(L):  # noqa: F811
    """Tokens times the query heads of a key head: at most 2**30."""
    assert attend(L, tokens=1 << 24, hq=2 * 65) == coc.ERR_SHAPE
    assert attend(L, _desc(kv_heads=1), tokens=(1 << 20) + 1, hq=1024) == coc.ERR_SHAPE
    assert attend(L, _desc(kv_heads=1), tokens=1 << 17, hq=65535) == coc.ERR_SHAPE
