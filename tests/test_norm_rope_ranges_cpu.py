"""Small outputs of norm and rotation in one pass (means, the weights' gradients) that overlap something else: every
call here fails on the host before anything is launched (no GPU needed)."""
import pytest

import block_sparse_attention_token_gb300 as sp
from tests.test_norm_rope_pass_cpu import FAKE, GAP, axes, call, lib, part  # noqa: F401

FREE = FAKE + 60 * GAP
OUT_Q, OUT_K = FAKE + 2 * GAP, FAKE + 10 * GAP
MEANS = 2 * 16 * 64 * 4           # bytes of means of 2 heads, 16 tiles


@pytest.mark.parametrize("q,k", [
    (dict(dw=FREE, db=FREE), None), (dict(dw=FREE, db=FREE + 240), None), (dict(dw=FREE), dict(dw=FREE)),
    (dict(db=FREE), dict(dw=FREE + 16)), (dict(dw=OUT_Q), None), (dict(db=OUT_K + 1024), {}), (dict(dw=FAKE), None),
    (dict(dw=FAKE + GAP), None), (dict(w=FREE, dw=FREE), None), ({}, dict(w=FREE, db=FREE - 240)), (dict(dw=FAKE - 4096), None),
    (dict(out=FAKE - 8192), None),
])
def test_backward(lib, q, k):
    assert call(lib, "bwd", q=part(0, **q), k=None if k is None else part(1, **k)) == sp.INVALID_ARG


@pytest.mark.parametrize("q,k,pos", [
    (dict(means=FREE), dict(means=FREE + MEANS - 16), None), (dict(means=FAKE), None, None), (dict(means=OUT_Q + 4096), None, None),
    ({}, dict(means=OUT_Q - MEANS + 16), None), (dict(b=FREE, means=FREE - 16), None, None), (dict(means=FREE), None, FREE + 16),
    (dict(out=FREE), None, FREE + 16), (dict(out=FREE, b=FREE + 64), None, None), (dict(means=FAKE - 4096), None, None),
])
def test_forward(lib, q, k, pos):
    assert call(lib, q=part(0, **q), k=None if k is None else part(1, **k), pos=pos) == sp.INVALID_ARG
