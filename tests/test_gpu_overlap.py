"""Calls that follow one another without a pause on one stream give the bits that they give one by one.

The attention may start before the projection in front of it has finished; it must not start before what is in
front of that projection has (a block boundary that writes the pools, a plan that writes the block table)."""
import pytest
import torch

from block_wise_kv_gb300 import dllm
from block_wise_kv_gb300.inputs import Workload, make_config
from block_wise_kv_gb300.step import LayerStep, block_rows_of, full_rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from block_wise_kv_gb300 import build

    build.build()
    dllm.load()
    torch.cuda.init()


def _graph(fn):
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


@pytest.mark.parametrize("name", ["mini", "wide"])
def test_boundary_projection_attention_in_one_graph(name):
    """The rows, and with them the cached states, differ from replay to replay; "wide" has the projection of many rows."""
    over = dict(t_prefix=[700, 90, 300], gen_len=[192, 256, 128], block=[32, 64, 16], block_index=[1, 0, 3], embedding=False)
    if name == "wide":
        over = dict(t_prefix=[700] * 6, gen_len=[192] * 6, block=[64] * 6, block_index=[1] * 6, embedding=False)
    cfg = make_config("tiny").with_(name=name, **over)
    wl = Workload(cfg)
    st = LayerStep(cfg, blocks=cfg.block_index, weights=wl.weights(0))
    x_full = full_rows_of(wl, 0, 0, cfg.block_index).cuda()
    x_block = block_rows_of(wl, 0, 0, cfg.block_index).cuda()

    def calls():
        st.boundary(x_full)
        st.step(x_block)

    graph = _graph(calls)
    for i in range(12):
        x_full.copy_(torch.randn(x_full.shape, device="cuda") * (1 + i % 3))
        x_block.copy_(torch.randn(x_block.shape, device="cuda"))
        st.boundary(x_full)
        torch.cuda.synchronize()
        st.qkv(x_block)
        torch.cuda.synchronize()
        st.step_attention()
        torch.cuda.synchronize()
        want = st.o_full.clone(), st.lse.clone()
        x_full.mul_(-1.0)  # other states in the pools before the replay
        st.boundary(x_full)
        x_full.mul_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert st.batch.error_bits() == 0
        assert torch.equal(st.o_full, want[0]) and torch.equal(st.lse, want[1]), i


def test_plan_projection_attention_in_one_graph():
    """The block table that the plan writes is the one that the attention behind the projection reads."""
    cfg = make_config("tiny").with_(name="planned", t_prefix=[500, 90, 300], gen_len=[128, 128, 128], block=[32, 32, 32],
                                    block_index=[1, 0, 2], embedding=False)
    wl = Workload(cfg)
    st = LayerStep(cfg, blocks=cfg.block_index, weights=wl.weights(0))
    x_full, x_block = full_rows_of(wl, 0, 0, cfg.block_index).cuda(), block_rows_of(wl, 0, 0, cfg.block_index).cuda()
    st.boundary(x_full)
    st.step(x_block)
    torch.cuda.synchronize()
    want = st.o_full.clone()
    t, c = st.batch.dev, st.batch.c
    held, out = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    pages = torch.cat([t["block_table"][b, :(n + 63) // 64] for b, n in enumerate(st.batch.host["seq_len"].tolist())])
    total = st.cache.num_pages
    ring_pages = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    ring_pages[:pages.numel()] = pages
    ring = dllm.PageRing(ring_pages, torch.tensor([0, pages.numel()], dtype=torch.int32, device="cuda"),
                         torch.zeros(2, dtype=torch.int32, device="cuda"))

    def calls():
        dllm.dllm_batch_plan(c, held, out, t["block_table"], t["cu_block"], t["cu_seq"], ring.c)
        st.step(x_block)

    graph = _graph(calls)
    for _ in range(10):
        t["block_table"].zero_()  # the plan has to put it back
        st.o_full.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert st.batch.error_bits() == 0
        assert torch.equal(st.o_full, want)
