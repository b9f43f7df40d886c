"""run_few_block refuses sizes as moe_layer_few does, with the same status, before it makes a workspace (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from combine_router_top_gb300 import build as B
    B.build()
    import combine_router_top_gb300 as M
    return M


@pytest.mark.parametrize("sizes,mlp,status", [
    (dict(T=33), dict(inner=256), "MOE_ERR_UNSUPPORTED"), (dict(H=264), dict(inner=256), "MOE_ERR_UNSUPPORTED"),
    (dict(), dict(inner=200), "MOE_ERR_UNSUPPORTED"), (dict(dtype=1), dict(inner=256), "MOE_ERR_UNSUPPORTED"),
    (dict(k=9), dict(inner=256), "MOE_ERR_INVALID_ARG"), (dict(), dict(inner=0), "MOE_ERR_INVALID_ARG"),
    (dict(), dict(inner=256, weights=2, group=16), "MOE_ERR_INVALID_ARG")])
def test_sizes(M, sizes, mlp, status):
    t, bufs = torch.zeros(64, dtype=torch.bfloat16), {}
    p = M.problem(**{**dict(T=4, H=256, E=8, k=2, R=1, Cap=4), **sizes})
    with pytest.raises(M.MoeError) as refusal:
        M.run_few_block(p, M.gate(), M.mlp(**mlp), M.norm(), *[t] * 11, bufs, t, t, t, stream=0)
    assert refusal.value.status == getattr(M, status) and not bufs
