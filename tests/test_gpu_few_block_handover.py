"""A block of a decode step on new inputs call after call, with nothing between the calls: each kernel of a call is launched
while the one before it still runs, so that a read ahead of its wait would find the call before's values. Two batches take
turns on one set of buffers; what each call leaves is copied away on its stream and compared with the same batch run alone."""
import pytest
import torch

from test_gpu_block_paths import DEV, M, make  # noqa: F401
from test_gpu_layer_few import make as make_layer

pytestmark = pytest.mark.gpu

INPUTS = ("x", "logits", "residual", "branch")
OUTPUTS = ("out", "r", "n")


@pytest.mark.parametrize("kind", ["bf16", "fp8", "w4"])
@pytest.mark.parametrize("T", [1, 7, 20, 32])
def test_two_batches_in_turn(M, T, kind):
    H, I, E, k = 1024, 512, 16, 4
    layer = make_layer(M, T, E, k, H, I, kind, 64, shared=1)
    s = make(M, T, "token")                              # the types of the join
    g = torch.Generator(device=DEV).manual_seed(3)
    w = [(1 + 0.2 * torch.randn(H, device=DEV, generator=g)).to(torch.bfloat16) for _ in range(2)]
    sets = [{"x": torch.randn((T, H), device=DEV, generator=g).to(torch.bfloat16),
             "logits": torch.randn((T, E), device=DEV, generator=g),
             "residual": 2.0 * torch.randn((T, H), device=DEV, generator=g),
             "branch": torch.rand(T, device=DEV, generator=g)} for _ in range(2)]
    now = {name: torch.empty_like(sets[0][name]) for name in INPUTS}
    made = {"out": torch.empty((T, H), dtype=torch.bfloat16, device=DEV), "r": torch.empty((T, H), device=DEV)}
    made["n"] = torch.empty_like(made["out"])
    bufs, p = {}, M.problem(T, H, E, k, 1, 1)

    def go(inputs, stream=None):
        M.run_few_block(p, layer["gate"], layer["mlp"], s["norm"], inputs["x"], inputs["logits"], layer["bias"],
                        layer["up"][0], layer["up"][1], layer["down"][0], layer["down"][1], inputs["residual"], *w,
                        inputs["branch"], bufs, made["out"], made["r"], made["n"], stream)
    want = []
    for inputs in sets:
        for v in made.values():
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        go(inputs)
        torch.cuda.synchronize()
        want.append({name: made[name].clone() for name in OUTPUTS})
    assert not any(torch.equal(want[0][name], want[1][name]) for name in OUTPUTS)
    got = []
    for i in range(24):                                  # inputs of their own, called straight behind one another
        go(sets[i % 2])
        if i % 3 == 2:
            got.append((i % 2, {name: made[name].clone() for name in OUTPUTS}))
    for i in range(24):                                  # the same input buffers, written anew between the calls
        for name in INPUTS:
            now[name].copy_(sets[i % 2][name])
        go(now)
        got.append((i % 2, {name: made[name].clone() for name in OUTPUTS}))
    torch.cuda.synchronize()
    assert M.moe_device_status() == M.MOE_OK
    for which, out in got:
        assert all(torch.equal(out[name], want[which][name]) for name in OUTPUTS)
