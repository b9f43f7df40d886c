"""The layer for a few tokens at the ends of its ranges: as many lists as there can be, the longest rows, tokens of every
magnitude, several calls at once. Tolerances as in test_gpu_layer_few."""
import pytest
import torch

from test_gpu_layer_few import DEV, KINDS, M, check, make, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("w4", 32), ("fp8", 128)])
def test_as_many_lists_as_pairs(M, kind, group):
    """32 tokens with 16 experts each, no expert twice, and the shared one: 513 lists."""
    s = make(M, 32, 1024, 16, 128, 128, kind, group, 1)
    s["bias"] = None
    for t in range(32):
        s["logits"][t, 16 * t:16 * t + 16] += 20.0
    s["gate"] = M.gate(M.MOE_SCORE_SIGMOID, scale=1.5)
    idx, w, out = run(M, s)
    assert idx.unique().numel() == 512
    check(s, idx, w, out)


def test_one_expert_for_all(M):
    """Every token's first choice is the last expert, whose list is as long as can be."""
    s = make(M, 32, 64, 3, 256, 384, "fp8", shared=1, sigmoid=False)
    s["logits"][:, 63] = 9.0
    check(s, *run(M, s))


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("w4", 64), ("fp8", 128)])
@pytest.mark.parametrize("T,H,I", [(2, 65536, 128), (9, 128, 65536)])
def test_longest_rows(M, T, H, I, kind, group):
    s = make(M, T, 2, 1, H, I, kind, group)
    check(s, *run(M, s))


@pytest.mark.parametrize("kind,group", KINDS)
def test_tokens_of_every_magnitude(M, kind, group):
    """Rows behind powers of two far apart, and one of zeros, in one batch; h then spans twice as many."""
    s = make(M, 12, 4, 2, 384, 256, kind, group, 1)
    for t, by in enumerate([2.0 ** 50, 2.0 ** -40, 0.0, 1.0, 2.0 ** 30, 2.0 ** -30, 2.0 ** 15, 2.0 ** -14]):
        s["x"][t] *= by
    idx, w, out = run(M, s)
    assert (out[2] == 0).all()
    check(s, idx, w, out)


def test_calls_at_once(M):
    """The same layer on three streams at once, each with an output and a workspace of its own."""
    s = make(M, 13, 16, 4, 1024, 640, "fp8", shared=1)
    _, _, want = run(M, s)
    p = M.problem(13, 1024, 16, 4, 1, 1)
    n = M.moe_layer_few_workspace_bytes(p, s["mlp"])
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in streams]
    spaces = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for stream, out, ws in zip(streams, outs, spaces):
            M.moe_layer_few(p, s["gate"], s["mlp"], s["x"], s["logits"], s["bias"], s["up"][0], s["up"][1], s["down"][0],
                            s["down"][1], None, None, out, ws, stream)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs) and M.moe_device_status() == M.MOE_OK
