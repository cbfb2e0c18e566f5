"""The kernel counts that Pipeline and attn_launches state, against those of the captured calls."""
import ctypes

import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_layer import COLS
from tests.test_gpu_masked import gen, masks

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

SMALL, SMALL64 = (1, 2, 4, 16, 16, 128, 2, 8, 8), (1, 2, 4, 16, 16, 64, 4, 4, 4)
LARGE, LARGE64 = (2, 3, 6, 32, 48, 128, 2, 8, 8), (1, 6, 8, 32, 32, 64, 4, 4, 4)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def kernels(run) -> int:
    """How many kernels one call launches: the kernel nodes of its capture (fills and copies are other nodes)."""
    cu = ctypes.CDLL("libcuda.so.1")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, n = ctypes.c_void_p(), ctypes.c_size_t()
    with torch.cuda.stream(side):
        run()                                       # memory and attributes are set up
        side.synchronize()
        assert cu.cuStreamBeginCapture_v2(ctypes.c_void_p(side.cuda_stream), 2) == 0      # relaxed
        run()
        assert cu.cuStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph)) == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    count, kind = 0, ctypes.c_int()
    for node in nodes:
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        count += kind.value == 0                    # CU_GRAPH_NODE_TYPE_KERNEL
    assert cu.cuGraphDestroy(graph) == 0
    return count


@pytest.mark.parametrize("dims", [SMALL, SMALL64, LARGE, LARGE64])
@pytest.mark.parametrize("kw", [
    {}, dict(flags=sp.SCHED_FLAT | sp.BWD_SPLIT_KV), dict(flags=sp.KERNEL_PORTABLE), dict(mask=True),
    dict(mask=True, cap=30.0), dict(cap=5.0), dict(mask=True, flags=sp.SCHED_FLAT | sp.BWD_SPLIT_KV),
    dict(mask=True, migrations=2, augment=True), dict(norm=True), dict(rope=True),
    dict(norm=True, rope=True, mask=True, cap=5.0), dict(norm=True, rope=True, flags=sp.KERNEL_PORTABLE),
    dict(raster_inputs=True), dict(raster_inputs=True, norm=True, rope=True, mask=True), dict(fused_estimation=False),
    dict(placement=True, gather=False), dict(estimator="lowrank", predictor_lr=0.0)],
    ids=lambda kw: "-".join(f"{k}={v}" for k, v in kw.items()) or "plain")
def test_pipeline_counts(dims, kw):
    s = sp.make_shape(*dims, "bf16")
    g = gen(71)
    kw = dict(kw)
    q, k, v, do = (torch.randn(s.B, s.N, s.H, s.d, generator=g, device="cuda").bfloat16() for _ in range(4))
    if kw.get("mask"):
        kw["mask"] = sp.mask_plan(s, *masks(s, "docs", g))
    if kw.get("norm"):
        kw["norm"] = sp.QKNorm(rms=True)
    if kw.get("rope"):
        kw["rope"] = sp.rope_table(s, COLS[s.d])
    backward = not kw.get("raster_inputs")
    w = {}
    if kw.get("estimator") == "lowrank":
        w = {x: torch.randn(s.H, s.d, 16, generator=g, device="cuda") for x in ("wq", "wk")}
    pipe = sp.Pipeline(s, kw.pop("estimator", "mean"), 0.5, 2, 2, backward=backward, **kw)
    assert kernels(lambda: pipe.forward(q, k, v, **w)) == pipe.kernels_per_forward()
    if backward:
        assert kernels(lambda: pipe.backward(do)) == pipe.kernels_per_backward()


@pytest.mark.parametrize("dims", [SMALL, SMALL64, LARGE, LARGE64])
@pytest.mark.parametrize("flags", [0, sp.LISTS_SEEN])
def test_call_counts(dims, flags):
    s = sp.make_shape(*dims, "bf16")
    g = gen(72)
    plan = sp.mask_plan(s, *masks(s, "docs", g))
    q, k, v = (torch.randn(s.B, s.H, s.N, s.d, generator=g, device="cuda").bfloat16() for _ in range(3))
    rp = torch.arange(s.rows + 1, device="cuda", dtype=torch.int32) * s.nb
    ci = torch.arange(s.nb, device="cuda", dtype=torch.int32).repeat(s.rows)
    for cap in (0.0, 5.0, 30.0):
        got = kernels(lambda: sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan, flags=flags))
        assert got == sp.attn_launches(s, False, True, cap, flags)
        o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan)
        got = kernels(lambda: sp.attn_masked_bwd(s, q, k, v, o, lse, v, rp, ci, cap=cap, mask=plan, flags=flags))
        assert got == sp.attn_launches(s, True, True, cap, flags)
