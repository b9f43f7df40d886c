"""Python binding of libmoe_gb300, the MoE route / dispatch / combine path on
one GB300 (sm_103a).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels, reached through ctypes with the same entry-point names as the C ABI in
``include/moe.h``. PyTorch supplies device memory and streams. There is no CPU
fallback: if the library is not built, or a tensor is not on a CUDA device,
the call raises.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_CUDA = -3
MOE_ERR_DEVICE_CHECK = -4
MOE_ERR_TIMEOUT = -5

MOE_DTYPE_BF16 = 0
MOE_DTYPE_FP8_E4M3_B128 = 1

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_GROUP_MAX = 0
MOE_GROUP_TOP2 = 1
MOE_LOGITS_F32 = 0
MOE_LOGITS_BF16 = 1
MOE_ACT_NONE = 0
MOE_ACT_SILU_GATE = 1

MOE_VALUE_BF16 = 0
MOE_VALUE_F32 = 1
MOE_BRANCH_PLAIN = 0
MOE_BRANCH_CHANNEL = 1
MOE_BRANCH_TOKEN = 2
MOE_WEIGHTS_BF16 = 0
MOE_WEIGHTS_FP8_B128 = 1
MOE_WEIGHTS_W4 = 2


class moe_problem(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("num_tokens", "hidden", "num_experts", "top_k", "num_ranks",
                                         "capacity", "dispatch_dtype", "max_blocks", "tokens_per_src_rank")]


class moe_gate(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("score", "num_groups", "top_groups", "group_rule", "renormalise",
                                         "logits_type")] + [("scale", C.c_float)]


class moe_w4(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_in", "n_out", "group", "act")]


class moe_norm(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("branch_gate", "residual_type", "param_type")] + \
        [(n, C.c_float) for n in ("eps", "scale")]


class moe_mlp(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("inner", "weights", "group", "shared")]


class moe_ubatch_bufs(C.Structure):
    _fields_ = [("topk_idx", C.c_void_p), ("topk_w", C.c_void_p), ("counts", C.c_void_p),
                ("offsets", C.c_void_p), ("slot", C.c_void_p), ("rank_counts", C.c_void_p),
                ("dropped", C.c_void_p), ("recv", C.c_void_p), ("recv_scale", C.c_void_p),
                ("recv_src", C.c_void_p), ("y", C.c_void_p), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t)]


class moe_dbo_timing(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("step_ms", "dispatch_ub1_ms", "combine_ub0_ms", "overlap_ms",
                                         "overlap_fraction")]


class moe_dbo_layers_args(C.Structure):
    _fields_ = [("full", moe_problem), ("n_layers", C.c_int32), ("busy_fmas", C.c_int32), ("alpha", C.c_float),
                ("sigma", C.c_float), ("x", C.c_void_p), ("logits", C.c_void_p), ("s", C.c_void_p),
                ("bufs", moe_ubatch_bufs * 2), ("h", C.c_void_p), ("shared", C.c_void_p), ("out", C.c_void_p),
                ("expert_w", C.c_void_p), ("mlp_max_blocks", C.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {moe_status_string(status)} ({status})")
        self.status = status


_lib = None


def lib() -> C.CDLL:
    """The loaded library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(LIB_PATH)
        P, i = C.c_void_p, C.c_int
        pp = C.POINTER(moe_problem)
        gp, wp = C.POINTER(moe_gate), C.POINTER(moe_w4)
        np_, mp = C.POINTER(moe_norm), C.POINTER(moe_mlp)
        sig = {
            "moe_status_string": ([i], C.c_char_p),
            "moe_validate": ([pp], i),
            "moe_device_status": ([], i),
            "moe_route_workspace_bytes": ([pp], C.c_size_t),
            "moe_route": ([pp, P, P, P, P, P, P, P, P, P, C.c_size_t, P], i),
            "moe_route_noalloc": ([pp, P, P, P, P, P, P, P, P, P], i),
            "moe_dispatch": ([pp, P, P, P, P, P, P, P], i),
            "moe_src_offsets": ([pp, P, P, P, P], i),
            "moe_route_dispatch_workspace_bytes": ([pp], C.c_size_t),
            "moe_route_dispatch": ([pp, P, P, P, P, P, P, P, P, P, P, P, P, P, C.c_size_t, P], i),
            "moe_expert_synthetic": ([pp, P, P, P, P, P, P], i),
            "moe_expert_gemm_fp8": ([pp, P, P, P, P, P, P, P], i),
            "moe_expert_gemm_bf16": ([pp, P, P, P, P, P], i),
            "moe_ready_flags_bytes": ([pp], C.c_size_t),
            "moe_path_host": ([pp, P, P, P, P, P, C.POINTER(moe_ubatch_bufs), P, P, P], i),
            "moe_expert_combine": ([pp, P, P, P, P, P, P, P, P, P, P, C.c_size_t, C.c_uint32, P], i),
            "moe_combine": ([pp, P, P, P, P, P, P], i),
            "moe_route_gated": ([pp, gp, P, P, P, P, P, P, P, P, P, P, C.c_size_t, P], i),
            "moe_route_gated_backward": ([pp, gp, P, P, P, P, P, P], i),
            "moe_combine_backward": ([pp, P, P, P, P, P, P, P, P], i),
            "moe_expert_w4_workspace_bytes": ([pp, wp], C.c_size_t),
            "moe_expert_w4": ([pp, wp, P, P, P, P, P, P, P, C.c_size_t, P], i),
            "moe_block_norm": ([pp, np_, P, P, P, P, P, P, P, P], i),
            "moe_combine_norm": ([pp, np_, P, P, P, P, P, P, P, P, P, P, P, P], i),
            "moe_block_norm_backward_workspace_bytes": ([pp, np_], C.c_size_t),
            "moe_block_norm_backward": ([pp, np_, P, P, P, P, P, P, P, P, P, P, P, P, P, C.c_size_t, P], i),
            "moe_layer_few_workspace_bytes": ([pp, mp], C.c_size_t),
            "moe_layer_few": ([pp, gp, mp, P, P, P, P, P, P, P, P, P, P, P, C.c_size_t, P], i),
            "dbo_create": ([C.POINTER(P)], i),
            "dbo_destroy": ([P], None),
            "dbo_step": ([P, pp, P, P, P, C.POINTER(moe_ubatch_bufs), P, P, P, i], i),
            "dbo_read_timing": ([P, C.POINTER(moe_dbo_timing)], i),
            "moe_layer_stand_in": ([P, P, C.c_int64, C.c_float, C.c_int32, P], i),
            "dbo_layers": ([P, C.POINTER(moe_dbo_layers_args), P, P], i),
            "dbo_layers_capture": ([P, C.POINTER(moe_dbo_layers_args), P, P], i),
            "dbo_graph_launch": ([P, P], i),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


EXPORTS = ("moe_status_string", "moe_validate", "moe_device_status", "moe_route_workspace_bytes", "moe_route", "moe_route_noalloc",
           "moe_dispatch", "moe_src_offsets", "moe_route_dispatch_workspace_bytes", "moe_route_dispatch",
           "moe_expert_synthetic", "moe_expert_gemm_fp8", "moe_expert_gemm_bf16", "moe_ready_flags_bytes", "moe_expert_combine", "moe_path_host",
           "moe_route_gated", "moe_route_gated_backward", "moe_combine_backward", "moe_expert_w4_workspace_bytes",
           "moe_expert_w4", "moe_block_norm", "moe_combine_norm", "moe_block_norm_backward_workspace_bytes",
           "moe_block_norm_backward", "moe_layer_few_workspace_bytes", "moe_layer_few",
           "moe_combine", "dbo_create", "dbo_destroy", "dbo_step", "dbo_read_timing",
           "moe_layer_stand_in", "dbo_layers", "dbo_layers_capture", "dbo_graph_launch")


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def problem(T, H, E, k, R, Cap, dtype=MOE_DTYPE_BF16, max_blocks=0, tokens_per_src_rank=0) -> moe_problem:
    return moe_problem(T, H, E, k, R, Cap, dtype, max_blocks, tokens_per_src_rank)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmoe_gb300 takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libmoe_gb300 takes contiguous tensors only")
    return t.data_ptr()


_raw_stream = None


def _stream(stream):
    global _raw_stream
    if stream is None:
        import torch
        if _raw_stream is None:
            # the current stream's handle without a Stream object around it: 0.3 instead of 3 us a call
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def moe_device_status() -> int:
    """MOE_OK, or MOE_ERR_TIMEOUT if a bounded device wait gave up since the last call (synchronises)."""
    return lib().moe_device_status()


def moe_validate(p: moe_problem) -> int:
    return lib().moe_validate(C.byref(p))


def moe_route_workspace_bytes(p: moe_problem) -> int:
    return lib().moe_route_workspace_bytes(C.byref(p))


def moe_route(p, logits, topk_idx, topk_w, counts, offsets, slot, rank_counts, dropped, workspace, stream=None):
    rc = lib().moe_route(C.byref(p), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                         _ptr(slot), _ptr(rank_counts), _ptr(dropped), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_route", rc)


def moe_route_noalloc(p, logits, topk_idx, topk_w, counts, offsets, slot, rank_counts, dropped, stream=None):
    """moe_route with the library's own static scratch instead of a workspace
    (for callers that cannot allocate device memory)."""
    rc = lib().moe_route_noalloc(C.byref(p), _ptr(logits), _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                                 _ptr(offsets), _ptr(slot), _ptr(rank_counts), _ptr(dropped), _stream(stream))
    _check("moe_route_noalloc", rc)


def src_ranks(p) -> int:
    """S, the number of virtual data-parallel source ranks of problem p."""
    T, tps = p.num_tokens, p.tokens_per_src_rank
    return max(1, (T + tps - 1) // tps) if tps > 0 else 1


def moe_src_offsets(p, counts, recv_src, src_offsets, stream=None):
    """src_offsets [E][S+1]: per expert, the first row of each source rank's tokens."""
    rc = lib().moe_src_offsets(C.byref(p), _ptr(counts), _ptr(recv_src), _ptr(src_offsets), _stream(stream))
    _check("moe_src_offsets", rc)


def moe_dispatch(p, x, topk_idx, slot, recv, recv_scale, recv_src, stream=None):
    rc = lib().moe_dispatch(C.byref(p), _ptr(x), _ptr(topk_idx), _ptr(slot), _ptr(recv), _ptr(recv_scale),
                            _ptr(recv_src), _stream(stream))
    _check("moe_dispatch", rc)


def moe_route_dispatch_workspace_bytes(p: moe_problem) -> int:
    return lib().moe_route_dispatch_workspace_bytes(C.byref(p))


def moe_route_dispatch(p, logits, x, topk_idx, topk_w, counts, offsets, slot, rank_counts, dropped, recv,
                       recv_scale, recv_src, workspace, stream=None):
    """moe_route then moe_dispatch in one call (fused into two launches for fp8 decode batches)."""
    rc = lib().moe_route_dispatch(C.byref(p), _ptr(logits), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                                  _ptr(offsets), _ptr(slot), _ptr(rank_counts), _ptr(dropped), _ptr(recv),
                                  _ptr(recv_scale), _ptr(recv_src), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_route_dispatch", rc)


def moe_expert_synthetic(p, recv, recv_scale, counts, s, y, stream=None):
    rc = lib().moe_expert_synthetic(C.byref(p), _ptr(recv), _ptr(recv_scale), _ptr(counts), _ptr(s), _ptr(y),
                                    _stream(stream))
    _check("moe_expert_synthetic", rc)


def moe_expert_gemm_fp8(p, recv_q, recv_scale, counts, w_q, w_scale, y, stream=None):
    """Grouped fp8 GEMM on the dispatch layout (tensor cores): y[e][r] = bf16(row . W_e^T) on kept rows."""
    rc = lib().moe_expert_gemm_fp8(C.byref(p), _ptr(recv_q), _ptr(recv_scale), _ptr(counts), _ptr(w_q),
                                   _ptr(w_scale), _ptr(y), _stream(stream))
    _check("moe_expert_gemm_fp8", rc)


def moe_expert_gemm_bf16(p, recv_x, counts, w, y, stream=None):
    """Grouped bf16 GEMM on the dispatch layout (tensor cores): y[e][r] = bf16(row . W_e^T) on kept rows."""
    rc = lib().moe_expert_gemm_bf16(C.byref(p), _ptr(recv_x), _ptr(counts), _ptr(w), _ptr(y), _stream(stream))
    _check("moe_expert_gemm_bf16", rc)


def moe_ready_flags_bytes(p: moe_problem) -> int:
    return lib().moe_ready_flags_bytes(C.byref(p))


def moe_expert_combine(p, recv, recv_scale, counts, s, y, topk_idx, topk_w, slot, out, flags, epoch: int,
                       stream=None):
    """Synthetic expert + combine in one kernel with per-row readiness flags (epoch: nonzero, fresh per call)."""
    rc = lib().moe_expert_combine(C.byref(p), _ptr(recv), _ptr(recv_scale), _ptr(counts), _ptr(s), _ptr(y),
                                  _ptr(topk_idx), _ptr(topk_w), _ptr(slot), _ptr(out), _ptr(flags),
                                  flags.numel() * flags.element_size(), epoch, _stream(stream))
    _check("moe_expert_combine", rc)


def moe_combine(p, y, topk_idx, topk_w, slot, out, stream=None):
    rc = lib().moe_combine(C.byref(p), _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(slot), _ptr(out),
                           _stream(stream))
    _check("moe_combine", rc)


def gate(score=MOE_SCORE_SOFTMAX, groups=1, top_groups=None, group_rule=MOE_GROUP_MAX, renormalise=True, scale=1.0,
         logits_type=MOE_LOGITS_F32) -> moe_gate:
    """How moe_route_gated chooses and weights; top_groups None: every group may be chosen from."""
    return moe_gate(score, groups, groups if top_groups is None else top_groups, group_rule, int(bool(renormalise)),
                    logits_type, scale)


def moe_route_gated(p, gate, logits, bias, topk_idx, topk_w, counts, offsets, slot, rank_counts, dropped, workspace,
                    stream=None):
    """moe_route with softmax or sigmoid scores, a balance bias (or None), groups and a scale on the weights."""
    rc = lib().moe_route_gated(C.byref(p), C.byref(gate), _ptr(logits), _ptr(bias), _ptr(topk_idx), _ptr(topk_w),
                               _ptr(counts), _ptr(offsets), _ptr(slot), _ptr(rank_counts), _ptr(dropped),
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_route_gated", rc)


def moe_route_gated_backward(p, gate, logits, topk_idx, topk_w, d_topk_w, d_logits, stream=None):
    """d_logits [T][E], every element written: the gradient of topk_w with the choice held fixed. logits may be
    None for a renormalised softmax."""
    rc = lib().moe_route_gated_backward(C.byref(p), C.byref(gate), _ptr(logits), _ptr(topk_idx), _ptr(topk_w),
                                        _ptr(d_topk_w), _ptr(d_logits), _stream(stream))
    _check("moe_route_gated_backward", rc)


def moe_combine_backward(p, y, d_out, topk_idx, topk_w, slot, d_y, d_topk_w, stream=None):
    """Gradient of moe_combine: d_y's rows of kept pairs (others are not written) and d_topk_w."""
    rc = lib().moe_combine_backward(C.byref(p), _ptr(y), _ptr(d_out), _ptr(topk_idx), _ptr(topk_w), _ptr(slot),
                                    _ptr(d_y), _ptr(d_topk_w), _stream(stream))
    _check("moe_combine_backward", rc)


def w4(n_in, n_out, group=128, act=MOE_ACT_NONE) -> moe_w4:
    """Shape of one 4-bit matrix per expert: n_out rows, or 2 n_out (gate, then up) for MOE_ACT_SILU_GATE."""
    return moe_w4(n_in, n_out, group, act)


def w4_pack(codes):
    """4-bit codes uint8 [..., K] (0..15, K a multiple of 128) in the inputs' order -> uint8 [..., K/2] as
    moe_expert_w4 reads them. Done once, when weights are loaded; any device."""
    import torch
    if codes.dtype != torch.uint8 or codes.shape[-1] % 128 != 0:
        raise ValueError("w4_pack takes uint8 codes, a multiple of 128 of them in the last dimension")
    c = codes.unflatten(-1, (-1, 4, 4, 4, 2))               # block, j, t, pair i, even or odd input
    c = c.transpose(-4, -3)                                  # block, t, j, i, even or odd
    halves = c.transpose(-2, -1)                             # ... even or odd, i: 4 codes to 16 bits
    return (halves[..., 0::2] | halves[..., 1::2] << 4).flatten(-5)


def w4_unpack(w_q):
    """The codes uint8 [..., K], in the inputs' order, of packed rows uint8 [..., K/2]."""
    import torch
    b = w_q.unflatten(-1, (-1, 4, 4, 2, 2))                  # block, t, j, even or odd, pair of codes
    halves = torch.stack([b & 15, b >> 4], -1).flatten(-2)   # ... even or odd, i
    return halves.transpose(-2, -1).transpose(-4, -3).flatten(-5)


def moe_expert_w4_workspace_bytes(p: moe_problem, w: moe_w4) -> int:
    return lib().moe_expert_w4_workspace_bytes(C.byref(p), C.byref(w))


def moe_expert_w4(p, w, x, x_scale, counts, w_q, w_scale, y, workspace, stream=None):
    """y[e][c] = x[e][c] . W_e^T (or its gated SiLU) on kept rows, W_e of 4-bit codes with group scales. x bf16 with
    x_scale None, or e4m3 codes with their scales, as p's dispatch type says."""
    rc = lib().moe_expert_w4(C.byref(p), C.byref(w), _ptr(x), _ptr(x_scale), _ptr(counts), _ptr(w_q), _ptr(w_scale),
                             _ptr(y), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_expert_w4", rc)


def norm(eps=1e-6, scale=1.0, gate=MOE_BRANCH_PLAIN, residual=MOE_VALUE_BF16, params=MOE_VALUE_BF16) -> moe_norm:
    """How a block's output joins the residual stream; residual and params: the types of its rows and of the weights."""
    return moe_norm(gate, residual, params, eps, scale)


def moe_block_norm(p, norm, y, residual, w_post, w_pre, gate, r, n, stream=None):
    """r = residual + scale * gate * N(y; w_post), n = N(r; w_pre) in one pass. w_post None: y as it is; y None: n of
    the residual alone; r or n may be left out (n together with w_pre)."""
    rc = lib().moe_block_norm(C.byref(p), C.byref(norm), _ptr(y), _ptr(residual), _ptr(w_post), _ptr(w_pre), _ptr(gate),
                              _ptr(r), _ptr(n), _stream(stream))
    _check("moe_block_norm", rc)


def moe_combine_norm(p, norm, y, topk_idx, topk_w, slot, residual, w_post, w_pre, gate, out, r, n, stream=None):
    """moe_combine and moe_block_norm in one pass; out (the combine's sum in bf16) may be None."""
    rc = lib().moe_combine_norm(C.byref(p), C.byref(norm), _ptr(y), _ptr(topk_idx), _ptr(topk_w), _ptr(slot),
                                _ptr(residual), _ptr(w_post), _ptr(w_pre), _ptr(gate), _ptr(out), _ptr(r), _ptr(n),
                                _stream(stream))
    _check("moe_combine_norm", rc)


def moe_block_norm_backward_workspace_bytes(p: moe_problem, norm: moe_norm) -> int:
    return lib().moe_block_norm_backward_workspace_bytes(C.byref(p), C.byref(norm))


def moe_block_norm_backward(p, norm, y, r, d_r, d_n, w_post, w_pre, gate, d_y, d_residual, d_w_post, d_w_pre, d_gate,
                            workspace, stream=None):
    """Gradient of moe_block_norm from y and the forward pass's r: d_y, d_residual, and where they are wanted the
    weights' and the gate's (f32). d_r None: no gradient reaches r directly."""
    rc = lib().moe_block_norm_backward(C.byref(p), C.byref(norm), _ptr(y), _ptr(r), _ptr(d_r), _ptr(d_n), _ptr(w_post),
                                       _ptr(w_pre), _ptr(gate), _ptr(d_y), _ptr(d_residual), _ptr(d_w_post),
                                       _ptr(d_w_pre), _ptr(d_gate), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_block_norm_backward", rc)


def mlp(inner, weights=MOE_WEIGHTS_BF16, group=128, shared=0) -> moe_mlp:
    """Shape of the experts' MLPs: H -> inner -> H; shared 1: one more expert, which every token has."""
    return moe_mlp(inner, weights, group, int(shared))


def moe_layer_few_workspace_bytes(p: moe_problem, mlp: moe_mlp) -> int:
    return lib().moe_layer_few_workspace_bytes(C.byref(p), C.byref(mlp))


def moe_layer_few(p, gate, mlp, x, logits, bias, w_up, up_scale, w_down, down_scale, topk_idx, topk_w, out, workspace,
                  stream=None):
    """The whole layer for up to 32 tokens in three or four launches: choice, gate and up products, SiLU, down product
    and weighted sum. Scales None for bf16 weights; topk_idx and topk_w may be None."""
    rc = lib().moe_layer_few(C.byref(p), C.byref(gate), C.byref(mlp), _ptr(x), _ptr(logits), _ptr(bias), _ptr(w_up),
                             _ptr(up_scale), _ptr(w_down), _ptr(down_scale), _ptr(topk_idx), _ptr(topk_w), _ptr(out),
                             _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("moe_layer_few", rc)


class DboContext:
    """Owns a moe_dbo_ctx (CUDA events only)."""

    def __init__(self):
        h = C.c_void_p()
        _check("dbo_create", lib().dbo_create(C.byref(h)))
        self.handle = h

    def close(self):
        if self.handle:
            lib().dbo_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dbo_create() -> DboContext:
    return DboContext()


def dbo_destroy(ctx: DboContext):
    ctx.close()


def ubatch_bufs(b: dict) -> moe_ubatch_bufs:
    """moe_ubatch_bufs from a dict of tensors laid out as alloc_buffers() makes them."""
    return moe_ubatch_bufs(_ptr(b["topk_idx"]), _ptr(b["topk_w"]), _ptr(b["counts"]), _ptr(b["offsets"]),
                           _ptr(b["slot"]), _ptr(b["rank_counts"]), _ptr(b["dropped"]), _ptr(b["recv"]),
                           _ptr(b.get("recv_scale")), _ptr(b["recv_src"]), _ptr(b["y"]), _ptr(b["workspace"]),
                           b["workspace"].numel() * b["workspace"].element_size())


def _host_ptr(t):
    if t.is_cuda:
        raise ValueError("moe_path_host takes host tensors for x_host, logits_host and out_host")
    if not t.is_contiguous():
        raise ValueError("libmoe_gb300 takes contiguous tensors only")
    return t.data_ptr()


class HostPath:
    """moe_path_host with its arguments marshalled once: every call() issues
    one batch (H2D of x and logits, the four stages, D2H of out) on `stream`."""

    def __init__(self, p: moe_problem, x_host, logits_host, s, x_dev, logits_dev, bufs: dict, out_dev, out_host,
                 stream=None):
        self.p = p
        self.ub = ubatch_bufs(bufs)
        self.args = (C.byref(self.p), _host_ptr(x_host), _host_ptr(logits_host), _ptr(s), _ptr(x_dev),
                     _ptr(logits_dev), C.byref(self.ub), _ptr(out_dev), _host_ptr(out_host), _stream(stream))
        self.fn = lib().moe_path_host
        self._keep = (x_host, logits_host, s, x_dev, logits_dev, bufs, out_dev, out_host)

    def __call__(self):
        _check("moe_path_host", self.fn(*self.args))


def moe_path_host(p, x_host, logits_host, s, x_dev, logits_dev, bufs: dict, out_dev, out_host, stream=None):
    """The whole path with host inputs and output, in one call (asynchronous on `stream`)."""
    HostPath(p, x_host, logits_host, s, x_dev, logits_dev, bufs, out_dev, out_host, stream)()


def dbo_step(ctx: DboContext, p_full, x, logits, s, bufs2, out, compute_stream, comm_stream, record_timing=False):
    arr = (moe_ubatch_bufs * 2)(ubatch_bufs(bufs2[0]), ubatch_bufs(bufs2[1]))
    rc = lib().dbo_step(ctx.handle, C.byref(p_full), _ptr(x), _ptr(logits), _ptr(s), arr, _ptr(out),
                        _stream(compute_stream), _stream(comm_stream), int(bool(record_timing)))
    _check("dbo_step", rc)


def dbo_read_timing(ctx: DboContext) -> dict:
    t = moe_dbo_timing()
    _check("dbo_read_timing", lib().dbo_read_timing(ctx.handle, C.byref(t)))
    return {n: getattr(t, n) for n, _ in moe_dbo_timing._fields_}


def alloc_buffers(p: moe_problem, device="cuda") -> dict:
    """Device buffers of every output of the path for problem p (torch.empty:
    contents undefined until written). Row buffers are bf16 stored as int16
    (or uint8 e4m3 codes)."""
    import torch
    T, H, E, k, R, Cap = p.num_tokens, p.hidden, p.num_experts, p.top_k, p.num_ranks, p.capacity
    fp8 = p.dispatch_dtype == MOE_DTYPE_FP8_E4M3_B128
    i32 = dict(dtype=torch.int32, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    ws = max(moe_route_workspace_bytes(p), moe_route_dispatch_workspace_bytes(p))
    if ws == 0:
        raise MoeError("moe_route_workspace_bytes", MOE_ERR_INVALID_ARG)
    b = {
        "topk_idx": torch.empty((T, k), **i32), "topk_w": torch.empty((T, k), **f32),
        "counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
        "slot": torch.empty((T, k), **i32), "rank_counts": torch.empty(R, **i32),
        "dropped": torch.empty(1, **i32),
        "recv": torch.empty((E, Cap, H), dtype=torch.uint8 if fp8 else torch.int16, device=device),
        "recv_scale": torch.empty((E, Cap, H // 128), **f32) if fp8 else None,
        "recv_src": torch.empty((E, Cap), **i32),
        "y": torch.empty((E, Cap, H), dtype=torch.int16, device=device),
        "workspace": torch.empty(ws, dtype=torch.uint8, device=device),
        # per-row readiness flags of moe_expert_combine: zero-filled once, then epoch-tagged
        "ready_flags": torch.zeros(max(moe_ready_flags_bytes(p) // 4, 1), **i32),
    }
    return b


def run_path(p: moe_problem, x, logits, s, bufs: dict, out, stream=None, fused=False):
    """route -> dispatch -> synthetic expert -> combine for one batch, on one stream
    (fused: route and dispatch through moe_route_dispatch)."""
    if fused:
        moe_route_dispatch(p, logits, x, bufs["topk_idx"], bufs["topk_w"], bufs["counts"], bufs["offsets"],
                           bufs["slot"], bufs["rank_counts"], bufs["dropped"], bufs["recv"], bufs.get("recv_scale"),
                           bufs["recv_src"], bufs["workspace"], stream)
    else:
        moe_route(p, logits, bufs["topk_idx"], bufs["topk_w"], bufs["counts"], bufs["offsets"], bufs["slot"],
                  bufs["rank_counts"], bufs["dropped"], bufs["workspace"], stream)
        moe_dispatch(p, x, bufs["topk_idx"], bufs["slot"], bufs["recv"], bufs.get("recv_scale"), bufs["recv_src"],
                     stream)
    moe_expert_synthetic(p, bufs["recv"], bufs.get("recv_scale"), bufs["counts"], s, bufs["y"], stream)
    moe_combine(p, bufs["y"], bufs["topk_idx"], bufs["topk_w"], bufs["slot"], out, stream)


def _w4_workspace(bufs: dict, n: int, device, stream: int, name="w4_workspace"):
    """bufs[name] of at least n bytes for work on the stream with this handle: made once, kept with the
    problem's buffers. Its memory belongs to the stream that it was made for, so that a dropped one is only handed on
    behind that stream's work; use on another stream is recorded with the allocator. One that a graph was captured with
    is kept beside it, in bufs[name + "_captured"], when a later call needs more: the graph writes to it at every replay."""
    import torch

    def torch_stream():                                  # ExternalStream takes no default stream
        return torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    ws = bufs.get(name)
    if ws is None or ws.numel() < n:
        with torch.cuda.stream(torch_stream()):
            bufs[name] = torch.empty(n, dtype=torch.uint8, device=device)
        bufs[name + "_stream"] = stream
    elif bufs.get(name + "_stream") != stream:
        ws.record_stream(torch_stream())
    if _capturing(stream, torch_stream):
        held = bufs.setdefault(name + "_captured", [])
        if not any(t is bufs[name] for t in held):
            held.append(bufs[name])


def _capturing(stream: int, torch_stream) -> bool:
    """Whether work on the stream with this handle, torch_stream() for torch, goes into a graph. 1 us for the current
    stream, 11 for another, which has to become the current one for the question."""
    import torch
    if not torch.cuda.is_initialized():
        return False
    if stream == _stream(None):
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(torch_stream()):
        return torch.cuda.is_current_stream_capturing()


def _w4_experts(p, gate, x, logits, bias, gate_up, down, b: dict, h, stream):
    """The steps of run_w4_path up to the experts' rows b["y"]."""
    T, H, E = p.num_tokens, p.hidden, p.num_experts
    pd = problem(T, H, E, p.top_k, p.num_ranks, p.capacity, MOE_DTYPE_BF16, p.max_blocks)     # h is bf16
    n = max(moe_expert_w4_workspace_bytes(p, gate_up[0]), moe_expert_w4_workspace_bytes(pd, down[0]))
    _w4_workspace(b, n, h.device, stream)
    moe_route_gated(p, gate, logits, bias, b["topk_idx"], b["topk_w"], b["counts"], b["offsets"], b["slot"],
                    b["rank_counts"], b["dropped"], b["workspace"], stream)
    moe_dispatch(p, x, b["topk_idx"], b["slot"], b["recv"], b.get("recv_scale"), b["recv_src"], stream)
    moe_expert_w4(p, gate_up[0], b["recv"], b.get("recv_scale"), b["counts"], gate_up[1], gate_up[2], h,
                  b["w4_workspace"], stream)
    moe_expert_w4(pd, down[0], h, None, b["counts"], down[1], down[2], b["y"], b["w4_workspace"], stream)


def run_w4_path(p: moe_problem, gate: moe_gate, x, logits, bias, gate_up, down, bufs: dict, h, out, stream=None):
    """moe_route_gated -> moe_dispatch -> experts with 4-bit weights (gate and up through SiLU, then down) ->
    moe_combine for one batch, on one stream. gate_up and down: (w4 shape, w_q, w_scale) of H -> I with
    MOE_ACT_SILU_GATE and of I -> H; bufs as alloc_buffers(p) makes them, to which the path adds the experts' workspace
    (which grows with the problem that needs more; one that a graph was captured with lives as long as bufs); h bf16
    [E][C][I], the MLP's inner rows."""
    b, stream = bufs, _stream(stream)
    _w4_experts(p, gate, x, logits, bias, gate_up, down, b, h, stream)
    moe_combine(p, b["y"], b["topk_idx"], b["topk_w"], b["slot"], out, stream)


def run_w4_block(p: moe_problem, gate: moe_gate, norm: moe_norm, x, logits, bias, gate_up, down, bufs: dict, h, residual,
                 w_post, w_pre, branch_gate, out, r, n, stream=None):
    """run_w4_path with its combine joined to the residual stream: r = residual + scale * branch_gate * N(y; w_post) and
    n = N(r; w_pre), the next block's input (moe_combine_norm). x is this block's input, the norm before it. out [T][H]
    bf16 keeps y for the way back (run_block_backward), or is None."""
    b, stream = bufs, _stream(stream)
    _w4_experts(p, gate, x, logits, bias, gate_up, down, b, h, stream)
    moe_combine_norm(p, norm, b["y"], b["topk_idx"], b["topk_w"], b["slot"], residual, w_post, w_pre, branch_gate, out, r, n,
                     stream)


def run_few_block(p: moe_problem, gate: moe_gate, mlp: moe_mlp, norm: moe_norm, x, logits, bias, w_up, up_scale, w_down,
                  down_scale, residual, w_post, w_pre, branch_gate, bufs: dict, out, r, n, stream=None):
    """A block of a decode step, for up to 32 tokens: moe_layer_few of x, this block's normed input, into out, then
    moe_block_norm of it with the residual stream into r and n, the next block's input. bufs: a dict of the caller's (empty
    at first) that keeps the layer's workspace, which grows with the problem that needs more; calls that may run at
    once, replayed graphs among them, have a dict each. A graph's workspace lives as long as the dict."""
    stream = _stream(stream)
    need = moe_layer_few_workspace_bytes(p, mlp)
    if need == 0:                                        # sizes that the layer refuses: with its own reason, nothing launched
        _check("moe_layer_few", lib().moe_layer_few(C.byref(p), C.byref(gate), C.byref(mlp), *[None] * 11, 0, None))
    _w4_workspace(bufs, need, x.device, stream, "few_workspace")
    moe_layer_few(p, gate, mlp, x, logits, bias, w_up, up_scale, w_down, down_scale, bufs.get("topk_idx"), bufs.get("topk_w"),
                  out, bufs["few_workspace"], stream)
    moe_block_norm(p, norm, out, residual, w_post, w_pre, branch_gate, r, n, stream)


def run_gate_backward(p: moe_problem, gate: moe_gate, logits, d_out, bufs: dict, d_y, d_topk_w, d_logits, stream=None):
    """The way back from moe_combine to the router: moe_combine_backward, then moe_route_gated_backward, on the
    buffers that a forward pass left. d_y [E][C][H] bf16 is the gradient of the experts' rows."""
    b = bufs
    moe_combine_backward(p, b["y"], d_out, b["topk_idx"], b["topk_w"], b["slot"], d_y, d_topk_w, stream)
    moe_route_gated_backward(p, gate, logits, b["topk_idx"], b["topk_w"], d_topk_w, d_logits, stream)


def run_block_backward(p: moe_problem, gate: moe_gate, norm: moe_norm, logits, out, r, d_r, d_n, w_post, w_pre, branch_gate,
                       bufs: dict, d_out, d_residual, d_w_post, d_w_pre, d_branch_gate, d_y, d_topk_w, d_logits, stream=None):
    """The way back through run_w4_block's join, combine and router: moe_block_norm_backward from the forward pass's out and
    r, then run_gate_backward of d_out, on the buffers that the forward pass left, to which it adds the norms' workspace as
    run_w4_path does the experts'. Weights' gradients may be None."""
    stream = _stream(stream)
    _w4_workspace(bufs, moe_block_norm_backward_workspace_bytes(p, norm), d_out.device, stream, "norm_workspace")
    moe_block_norm_backward(p, norm, out, r, d_r, d_n, w_post, w_pre, branch_gate, d_out, d_residual, d_w_post, d_w_pre,
                            d_branch_gate, bufs["norm_workspace"], stream)
    run_gate_backward(p, gate, logits, d_out, bufs, d_y, d_topk_w, d_logits, stream)


def moe_layer_stand_in(x, out, a: float, busy_fmas: int = 0, stream=None):
    """out = bf16(x * a) (+ busy work that does not change the output)."""
    _check("moe_layer_stand_in", lib().moe_layer_stand_in(_ptr(x), _ptr(out), x.numel(), float(a), int(busy_fmas),
                                                          _stream(stream)))


def dbo_layers_args(p_full, n_layers, x, logits, s, bufs2, h, shared, out, alpha=1.0, sigma=1.0, busy_fmas=0,
                    expert_w=None, mlp_max_blocks=0):
    """moe_dbo_layers_args from tensors (the struct keeps raw pointers: keep the tensors alive).
    expert_w: [E][H][H] bf16 weights for the grouped GEMM as the MLP, or None for the synthetic expert."""
    a = moe_dbo_layers_args()
    a.full = p_full
    a.n_layers, a.busy_fmas, a.alpha, a.sigma = int(n_layers), int(busy_fmas), float(alpha), float(sigma)
    a.x, a.logits, a.s = _ptr(x), _ptr(logits), _ptr(s)
    a.bufs[0], a.bufs[1] = ubatch_bufs(bufs2[0]), ubatch_bufs(bufs2[1])
    a.h, a.shared, a.out = _ptr(h), _ptr(shared), _ptr(out)
    a.expert_w, a.mlp_max_blocks = _ptr(expert_w), int(mlp_max_blocks)
    return a


def dbo_layers(ctx: DboContext, args, compute_stream, comm_stream):
    _check("dbo_layers", lib().dbo_layers(ctx.handle, C.byref(args), _stream(compute_stream), _stream(comm_stream)))


def dbo_layers_capture(ctx: DboContext, args, compute_stream, comm_stream):
    _check("dbo_layers_capture", lib().dbo_layers_capture(ctx.handle, C.byref(args), _stream(compute_stream),
                                                          _stream(comm_stream)))


def dbo_graph_launch(ctx: DboContext, stream=None):
    _check("dbo_graph_launch", lib().dbo_graph_launch(ctx.handle, _stream(stream)))
