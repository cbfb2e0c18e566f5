"""Rows handed to the cache's calls: strides that are read as they are, and broadcast views, which are refused (no GPU
needed)."""
import pytest

import block_sparse_attention_token_gb300 as sp
from block_sparse_attention_token_gb300.cache import _rows

torch = pytest.importorskip("torch")
CPU = -1   # the device number of a tensor in host memory


@pytest.mark.parametrize("shape,to", [((6, 1, 64), (6, 3, 64)), ((1, 3, 64), (6, 3, 64)), ((1, 1, 64), (6, 3, 64)),
                                      ((1, 1, 64), (6, 1, 64)), ((1, 1, 64), (1, 3, 64)), ((6, 3, 1), (6, 3, 64))])
def test_broadcast_views_are_refused(shape, to):
    with pytest.raises(ValueError):
        _rows("k", torch.randn(shape).expand(to), to[1], to[2], CPU)


def test_strides_as_they_are():
    wide = torch.randn(6, 8, 64)
    t = wide[:, 2:5]
    assert _rows("k", t, 3, 64, CPU, 6) == (t.data_ptr(), 512, 64)
    t = torch.randn(3, 6, 64).transpose(0, 1)                  # tile order
    assert _rows("k", t, 3, 64, CPU) == (t.data_ptr(), 64, 384)
    t = wide[::2, ::4]
    assert _rows("k", t, 2, 64, CPU) == (t.data_ptr(), 1024, 256)
    # a stride over one token or one head says nothing: also that of a view expanded to its own size
    t = wide[:1, :3]
    assert _rows("k", t, 3, 64, CPU) == (t.data_ptr(), 0, 64)
    t = torch.randn(1, 1, 64).expand(1, 1, 64)
    assert _rows("k", t, 1, 64, CPU) == (t.data_ptr(), 0, 0)
    t = torch.randn(1, 3, 64).expand(0, 3, 64)                 # no tokens
    assert _rows("k", t, 3, 64, CPU)[1:] == (0, 64)
    for bad in (wide.transpose(1, 2), wide[0], wide[:, :2], wide[:, :3, :32], wide[..., ::2]):
        with pytest.raises(ValueError):
            _rows("k", bad, 3, 64, CPU)


@pytest.mark.gpu
@pytest.mark.timeout(300)
@pytest.mark.parametrize("to", [(6, 3, 64), (1, 3, 64), (6, 1, 64)])
def test_calls_refuse_broadcast_views(to):
    """Keys, values or queries of one head or token given to several: an error before anything runs, and what a copy
    of the view gives is what the rows say."""
    import __graft_entry__
    __graft_entry__.build()
    n, heads, d = to
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = sp.block_pool(2, heads, d, 64)
    before = [t.view(torch.uint8).clone() for t in (pool.k, pool.v)]
    slots = torch.arange(n, **i32)
    dense = torch.randn(n, heads, d, device="cuda")
    args = torch.tensor([0, n], **i32), torch.tensor([n], **i32), torch.zeros(1, 1, **i32), n
    for one in ((n, 1, d), (1, heads, d), (1, 1, d)):
        if one == to:
            continue
        view = torch.randn(one, device="cuda").expand(to)
        for k, v in ((view, dense), (dense, view)):
            with pytest.raises(ValueError):
                sp.cache_write(pool, k, v, slots)
        with pytest.raises(ValueError):
            sp.attn_cache_fwd(pool, view.bfloat16().contiguous()[:1, :1].expand(to), *args)
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (pool.k, pool.v)))
    view = torch.randn(n, 1, d, device="cuda").expand(to).contiguous()
    sp.cache_write(pool, view, view.clone(), slots)
    got = pool.k[0, :, :n].float() * pool.k_scale[0][:, None, None]
    assert ((got - view.transpose(0, 1)).abs() <= 2.0 ** -4 * view.transpose(0, 1).abs() + 2.0 ** -10 * view.abs().max()).all()
