"""Arguments of the cache's calls that overlap in part: every call here fails on the host before anything is launched
(no GPU needed)."""
import pytest

import block_sparse_attention_token_gb300 as sp
from tests.test_cache_cpu import FAKE, GAP, at, attn, cache, lib, write  # noqa: F401

CODES, SCALES = 10 * 2 * 64 * 64, 4 * 10 * 2    # bytes of the pools of cache()
ROWS = 5 * 2 * 64 * 2                           # bytes of packed k and v


@pytest.mark.parametrize("kw", [
    dict(vc=at(3) + CODES - 16), dict(kc=at(5) + CODES - 16), dict(vsc=at(4) + SCALES - 16), dict(ksc=at(3) + 4096),
    dict(vsc=at(3) + CODES - 16), dict(kc=at(6) - CODES + 16), dict(ksc=at(5)),
    dict(slots=at(3) + 16), dict(slots=at(4)), dict(slots=at(6) - 16), dict(slots=at(5) + CODES - 16),
    dict(k=at(3)), dict(k=at(3) - ROWS + 16), dict(v=at(5) + CODES - 16), dict(v=at(4)), dict(k=at(6) - 16),
    dict(k=at(3) - 4096 - 64 * 2, ks=1024 + 64),            # its last token's row only
    dict(v=at(5) - 4096, vh=2048),                       # its last head only
    dict(dtype=sp.F32, k=at(3) - 2 * ROWS + 16),
])
def test_write_refuses_overlaps(lib, kw):
    assert write(lib, **kw) == sp.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(ks=1 << 40, tokens=(1 << 31) - 1), dict(vs=1 << 40, tokens=1 << 22)])
def test_write_refuses_rows_beyond_any_memory(lib, kw):
    assert write(lib, **kw) == sp.SHAPE


@pytest.mark.parametrize("kw", [
    dict(o=at(4)), dict(o=at(4) + CODES - 16), dict(lse=at(5)), dict(lse=at(6) + 4096), dict(o=at(7) + SCALES - 16),
    dict(lse=at(1)), dict(lse=at(2)), dict(o=at(3) - 16), dict(lse=at(11), row_ptr=at(11), col_idx=at(12), col_cap=9),
    dict(o=at(12) + 32, row_ptr=at(11), col_idx=at(12), col_cap=9),
    dict(o=at(12) + (1 << 30), row_ptr=at(11), col_idx=at(12), col_cap=1 << 62),
])
def test_attn_refuses_overlaps(lib, kw):
    assert attn(lib, **kw) == sp.INVALID_ARG
