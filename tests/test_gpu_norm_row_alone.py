"""A row's r and n depend on its own values alone: the same bits whatever else is in the batch, however many rows there are
and whichever kernel they take. The sizes stand on both sides of every limit at which the number of rows or the row's length
chooses a kernel: 608 rows and 8192 channels (moe_block_norm), 304 tokens and 2048 channels (moe_combine_norm)."""
import pytest
import torch

from test_gpu_block_norm import DEV, M, check_forward, forward, make, routing  # noqa: F401

pytestmark = pytest.mark.gpu

WIDTHS = [8, 264, 2048, 2056, 2304, 4096, 4104, 5128, 7168, 7176, 8192, 8200, 16384]
FORMS = [("none", "bf16", "bf16", True, True), ("channel", "f32", "bf16", True, True), ("token", "bf16", "f32", False, True),
         ("channel", "bf16", "f32", True, False)]


def rows_of(s, at):
    """The rows `at` of a batch as a batch of their own."""
    t = {**s, "T": len(at)}
    for name in ("y", "residual"):
        t[name] = s[name][at].contiguous()
    if s["kind"] == "token":
        t["gate"] = s["gate"][at].contiguous()
    return t


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("kind,res,par,post,pre", FORMS)
def test_block_norm(M, H, kind, res, par, post, pre):
    s = make(M, 640, H, kind, res, par, post, pre)
    r, n = forward(M, s)
    check_forward(s, r, n)
    for at in ([639], [0, 5], list(range(607)), list(range(32, 640))):
        t = rows_of(s, at)
        r2, n2 = forward(M, {**t, "p": M.problem(len(at), H, 1, 1, 1, 1)})
        assert torch.equal(r2, r[at])
        assert n is None or torch.equal(n2, n[at])


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("kind,res,par,post,pre", FORMS)
def test_combine_norm(M, H, kind, res, par, post, pre):
    T, E, k, C = 320, 16, 5, 60
    s = make(M, T, H, kind, res, par, post, pre)
    idx, w, slot, _ = routing(M, T, E, k, C, T + H, {3, 319})
    g = torch.Generator(device=DEV).manual_seed(7)
    y = torch.randn((E, C, H), device=DEV, generator=g).to(torch.bfloat16)

    def go(at):
        t = rows_of(s, at)
        out = torch.full((len(at), H), float("nan"), dtype=torch.bfloat16, device=DEV)
        r, n = torch.full_like(t["residual"], float("nan")), torch.full_like(out, float("nan")) if pre else None
        rows = [v[at].contiguous() for v in (idx, w, slot)]
        M.moe_combine_norm(M.problem(len(at), H, E, k, 1, C), s["norm"], y, *rows, t["residual"], s["w_post"], s["w_pre"],
                           t["gate"], out, r, n)
        torch.cuda.synchronize()
        assert M.moe_device_status() == M.MOE_OK
        return [v for v in (out, r, n) if v is not None]
    whole = go(list(range(T)))
    assert all(torch.isfinite(v.float()).all() for v in whole)
    for at in ([319], [7], [0, 5], list(range(303)), list(range(16, 320))):
        assert all(torch.equal(a, b[at]) for a, b in zip(go(at), whole))
