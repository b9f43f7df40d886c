"""Who owns run_w4_path's workspace: it is made for the stream that the kernels run on, and a later call on another
stream records its use, so that the allocator hands its memory on only behind the work that reads it. The first test
stands in for the streams and the kernels on the CPU; the second grows a real one behind unfinished work."""
import contextlib

import pytest
import torch

import combine_router_top_gb300 as M


@pytest.fixture(scope="module")
def built():
    from combine_router_top_gb300 import build as B
    B.build()


def fp8_path(E=4, C=32, H=128):
    """Problems whose experts have many rows: the workspace holds the rows as fp16."""
    w = M.w4(H, H, 64)
    return lambda T, C=C: M.problem(T, H, E, 2, 1, C, M.MOE_DTYPE_FP8_E4M3_B128), w


def test_the_workspace_belongs_to_the_callers_stream(built, monkeypatch):
    problem, w = fp8_path()
    active, made, recorded, used = [7], [], [], []

    @contextlib.contextmanager
    def on(s):
        active.append(int(s))
        yield
        active.pop()
    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(M, "_raw_stream", lambda device: 7)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(active[-1]) or empty(*a, **k))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), int(s))))
    for f in ("moe_route_gated", "moe_dispatch", "moe_combine"):
        monkeypatch.setattr(M, f, lambda *a: None)
    monkeypatch.setattr(M, "moe_expert_w4", lambda *a: used.append(a[8].data_ptr()))
    b = dict.fromkeys(("topk_idx", "topk_w", "counts", "offsets", "slot", "rank_counts", "dropped", "recv", "recv_src",
                       "y", "workspace"))
    h = empty(1)

    def path(T, stream, C=32):
        M.run_w4_path(problem(T, C), M.gate(), None, None, None, (w, None, None), (w, None, None), b, h, None, stream)
    path(40, 11)
    assert made == [11]                                 # made on the stream that its kernels run on
    path(40, 11)
    assert made == [11] and not recorded                # kept
    path(40, 12)
    assert recorded == [(b["w4_workspace"].data_ptr(), 12)]
    path(40, 13, C=64)                                  # more than there is: another one, on its own stream
    assert made == [11, 13]
    path(40, None, C=128)                               # the current stream
    path(40, 0, C=256)                                  # the default stream
    assert made == [11, 13, 7, 0] and len(recorded) == 1
    assert used[-1] == used[-2] == b["w4_workspace"].data_ptr()


@pytest.mark.gpu
def test_a_larger_problem_on_a_side_stream_leaves_the_earlier_calls_rows_alone(built):
    """Two problems on a stream of their own, the second with more rows, while the current stream takes and overwrites
    memory of the first one's size: nothing waits between the calls."""
    dev, H, E = "cuda:0", 128, 4
    problem, w = fp8_path(E, 32, H)
    g = torch.Generator(device=dev).manual_seed(1)
    weights = (w, torch.randint(0, 256, (E, H, H // 2), dtype=torch.uint8, device=dev, generator=g),
               torch.full((E, H, H // 64), 0.02, dtype=torch.bfloat16, device=dev))
    x = torch.randn((40, H), device=dev, generator=g).to(torch.bfloat16)
    logits = torch.randn((40, E), device=dev, generator=g)
    sizes = (32, 96)
    bufs = {C: M.alloc_buffers(problem(40, C), dev) for C in sizes}
    h = {C: torch.empty((E, C, H), dtype=torch.bfloat16, device=dev) for C in sizes}
    out = {C: torch.empty((40, H), dtype=torch.bfloat16, device=dev) for C in sizes}

    def path(C, o, stream):
        M.run_w4_path(problem(40, C), M.gate(), x, logits, None, weights, weights, bufs[C], h[C], o, stream)
    for C in sizes:
        path(C, out[C], None)
    torch.cuda.synchronize()
    got = {C: torch.empty_like(out[C]) for C in sizes}
    n = M.moe_expert_w4_workspace_bytes(problem(40, sizes[0]), w)
    assert n > 256
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        for b in bufs.values():
            b.pop("w4_workspace", None)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.ExternalStream(M._stream(stream))):
            torch.cuda._sleep(100_000_000)              # the work below is queued behind about 50 ms
        path(sizes[0], got[sizes[0]], stream)
        old = bufs[sizes[0]].pop("w4_workspace")
        at = old.data_ptr()
        bufs[sizes[1]]["w4_workspace"] = old            # outgrown, and dropped, by the next call
        del old
        path(sizes[1], got[sizes[1]], stream)
        taken = [torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(64)]
        assert all(not t.data_ptr() <= at < t.data_ptr() + n for t in taken)
        torch.cuda.synchronize()
        for C in sizes:
            assert torch.equal(got[C], out[C])
