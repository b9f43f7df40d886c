"""The layer for a few tokens where several blocks share the down product's outputs: a grid so small that a block takes one
unit after another, one workspace for call after call, and a replayed graph. The same bits every time, and within the
bounds of test_gpu_layer_few of the plain form.

How many blocks share a unit is set by the sizes: 2 at 2048 outputs of 1408 inputs with 25 experts' rows, 8 at 128 outputs
of 65 536 inputs with 2, and 4 (4-bit weights) or 8 at 256 of 32 768."""
import pytest
import torch

from test_gpu_layer_few import DEV, M, check, make  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(13, 24, 4, 2048, 1408, 1), (9, 2, 1, 128, 65536, 0), (5, 2, 2, 256, 32768, 0)]


def call(M, s, ws, out, stream=None, max_blocks=0):
    p = M.problem(s["T"], s["H"], s["E"], s["k"], 1, 1, max_blocks=max_blocks)
    M.moe_layer_few(p, s["gate"], s["mlp"], s["x"], s["logits"], s["bias"], s["up"][0], s["up"][1], s["down"][0], s["down"][1],
                    None, None, out, ws, stream)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "w4"])
@pytest.mark.parametrize("T,E,k,H,I,shared", SHAPES)
def test_units_in_turn_and_calls_in_a_row(M, T, E, k, H, I, shared, kind):
    s = make(M, T, E, k, H, I, kind, 128, shared)
    n = M.moe_layer_few_workspace_bytes(M.problem(T, H, E, k, 1, 1), s["mlp"])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    want = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    call(M, s, ws, want)
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    check(s, None, None, want)
    for blocks in (1, 5, 40, 0, 0):                      # the workspace as the call before left it
        out = torch.full_like(want, float("nan"))
        call(M, s, ws, out, max_blocks=blocks)
        torch.cuda.synchronize()
        assert M.moe_device_status() == M.MOE_OK
        assert torch.equal(out, want), blocks
    # several calls with nothing between them, captured and replayed
    outs = [torch.full_like(want, float("nan")) for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for out, blocks in zip(outs, (0, 5, 0)):
            call(M, s, ws, out, side, blocks)
    for _ in range(2):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)
    assert M.moe_device_status() == M.MOE_OK
