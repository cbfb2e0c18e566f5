"""Refusals of the list compaction under a token mask, on the host (no GPU needed)."""
import ctypes

import pytest

import block_sparse_attention_token_gb300 as sp

FAKE, GAP = 1 << 20, 1 << 24


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_token_gb300 import build
    build.build()
    return sp.lib()


def test_mask_csr_refuses(lib):
    s = sp.make_shape(1, 2, 4, 16, 16, 64, 4, 4, 4, sp.BF16)

    def call(sh=s, plan=FAKE, rp=FAKE, ci=FAKE, rp2=FAKE + GAP, ci2=FAKE + GAP, status=None):
        return lib.sparsp_mask_csr(ctypes.byref(sh), plan, rp, ci, rp2, ci2, status, None)
    for name in ("plan", "rp", "ci", "rp2", "ci2"):
        assert call(**{name: None}) == sp.INVALID_ARG
        assert call(**{name: FAKE + 4}) == sp.ALIGN
    assert call(status=FAKE + 4) == sp.ALIGN
    assert call(rp2=FAKE) == sp.INVALID_ARG and call(rp2=FAKE + 16) == sp.INVALID_ARG
    assert call(ci2=FAKE) == sp.INVALID_ARG
    assert call(sh=sp.make_shape(1, 2, 5, 16, 16, 64, 4, 4, 4, sp.BF16)) == sp.SHAPE
    assert lib.sparsp_attn_masked_compacts(ctypes.byref(sp.make_shape(0, 2, 4, 16, 16, 64, 4, 4, 4, sp.BF16)), 0) == 0


def test_plain_attention_ignores_the_lists_option(lib):
    s = sp.make_shape(1, 2, 4, 16, 16, 64, 4, 4, 4, sp.BF16)
    args = (FAKE,) * 5
    call = lambda flags: lib.sparsp_attn_fwd(ctypes.byref(s), *args, 0.0, FAKE, FAKE, FAKE, 16, flags, None, None, None)
    assert call(sp.LISTS_SEEN) == sp.WORKSPACE      # a known option: the call goes on to the workspace's size
    assert call(1 << 6) == sp.INVALID_ARG
