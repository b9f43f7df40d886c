"""A workspace that the package keeps with a caller's buffers stays where a captured graph writes to it, when a later call
on the same buffers needs a larger one. The first test stands in for the allocator and the streams on the CPU; the second
replays such a graph."""
import contextlib

import pytest
import torch

import combine_router_top_gb300 as M


@pytest.fixture(scope="module")
def built():
    from combine_router_top_gb300 import build as B
    B.build()


@pytest.mark.parametrize("name", ["w4_workspace", "few_workspace", "norm_workspace"])
def test_a_captured_workspace_is_kept(built, monkeypatch, name):
    capturing = set()
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(M, "_capturing", lambda stream, torch_stream: stream in capturing, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    b = {}

    def use(n, stream):
        M._w4_workspace(b, n, "cpu", stream, name)
        return b[name].data_ptr()

    def kept():
        return [t.data_ptr() for t in b.get(name + "_captured", [])]
    use(100, 7)
    assert kept() == []                                  # eager calls keep one only
    use(200, 7)
    assert kept() == [] and b[name].numel() == 200
    capturing.add(11)
    first = use(200, 11)
    assert use(150, 11) == first and kept() == [first]   # once, whatever the number of calls
    capturing.clear()
    second = use(300, 7)
    assert second != first and kept() == [first]         # outgrown, and still there
    capturing.add(7)
    assert use(300, 7) == second and kept() == [first, second]


@pytest.mark.gpu
def test_a_larger_call_leaves_a_graph_its_workspace(built):
    """The way back of 8 tokens captured, then run for 400 on the same buffers, then memory taken in sizes of the first
    workspace: replays of the graph give what they gave, and write to none of that memory."""
    dev, H, E, k, C = "cuda:0", 512, 8, 2, 128
    g = torch.Generator(device=dev).manual_seed(1)
    T = 400
    p = {n: M.problem(n, H, E, k, 1, C) for n in (8, T)}
    norm, gate = M.norm(residual=M.MOE_VALUE_F32), M.gate()
    b = M.alloc_buffers(p[T], dev)
    f32 = dict(dtype=torch.float32, device=dev)
    bf = dict(dtype=torch.bfloat16, device=dev)
    logits = torch.randn((T, E), device=dev, generator=g)
    out, d_n = (torch.randn((T, H), device=dev, generator=g).to(torch.bfloat16) for _ in range(2))
    r, d_r = (torch.randn((T, H), device=dev, generator=g) for _ in range(2))
    w_post, w_pre = torch.ones(H, **bf), torch.ones(H, **bf)
    b["y"].view(torch.bfloat16).normal_(generator=g)
    made = dict(d_out=torch.empty((T, H), **bf), d_res=torch.empty((T, H), **f32), d_post=torch.empty(H, **f32),
                d_pre=torch.empty(H, **f32), d_y=torch.zeros((E, C, H), **bf), d_w=torch.empty((T, k), **f32),
                d_l=torch.empty((T, E), **f32))

    def go(n, stream=None):
        M.run_block_backward(p[n], gate, norm, logits[:n], out[:n], r[:n], d_r[:n], d_n[:n], w_post, w_pre, None, b,
                             made["d_out"][:n], made["d_res"][:n], made["d_post"], made["d_pre"], None, made["d_y"],
                             made["d_w"][:n], made["d_l"][:n], stream)

    def route(n):
        M.moe_route_gated(p[n], gate, logits[:n], None, b["topk_idx"], b["topk_w"], b["counts"], b["offsets"], b["slot"],
                          b["rank_counts"], b["dropped"], b["workspace"])
    route(8)
    go(8)
    torch.cuda.synchronize()
    want = {n: made[n].clone() for n in ("d_post", "d_pre")}
    size, at = b["norm_workspace"].numel(), b["norm_workspace"].data_ptr()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        go(8)
    assert [t.data_ptr() for t in b["norm_workspace_captured"]] == [at]
    route(T)
    go(T)
    torch.cuda.synchronize()
    assert b["norm_workspace"].numel() > size and b["norm_workspace"].data_ptr() != at
    taken = [torch.full((size,), 0x5A, dtype=torch.uint8, device=dev) for _ in range(64)]
    assert all(not t.data_ptr() <= at < t.data_ptr() + size for t in taken)
    route(8)
    for _ in range(2):
        for n in want:
            made[n].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(made[n], v) for n, v in want.items())
    assert all((t == 0x5A).all() for t in taken) and M.moe_device_status() == M.MOE_OK
