"""Performance cases of the gated route, its gradient, the combine's gradient and the experts' products with 4-bit
weights.

    route            moe_route_gated: softmax or sigmoid scores, a balance bias, groups, top-k, renormalised weights,
                     then counts, offsets and slots as moe_route gives them
    route_backward   moe_route_gated_backward: the gradient of the routing weights with respect to the logits
    combine_backward moe_combine_backward: the gradients of the weighted sum with respect to the experts' rows and to
                     the routing weights
    expert_w4        moe_expert_w4: rows of each expert times that expert's 4-bit matrix with group scales, as they
                     are or through the gated SiLU

Each case is run in a plain form (elementary torch operations in 32 bits, rounded once at the end) or, where `own` is
set, by the calls of the package.
"""
import math

import torch

own = False

DEV = "cuda"


# ---- cases ----------------------------------------------------------------------------------------------------------

def _route(name, T, E, k, R, C, score="sigmoid", bias=True, G=1, top_g=1, rule="max", renorm=True, scale=1.0,
           logits="f32"):
    c = {"op": "route", "T": T, "E": E, "k": k, "R": R, "C": C, "score": score, "bias": bias, "G": G, "top_g": top_g,
         "rule": rule, "renorm": renorm, "scale": scale, "logits": logits}
    return {"name": name, **c} if name else c


def _combine(name, T, H, E, k, C):
    c = {"op": "combine_backward", "T": T, "H": H, "E": E, "k": k, "C": C}
    return {"name": name, **c} if name else c


def _w4(name, T, E, k, C, n_in, n_out, group=128, act="none", x="bf16"):
    c = {"op": "expert_w4", "T": T, "E": E, "k": k, "C": C, "n_in": n_in, "n_out": n_out, "group": group, "act": act,
         "x": x}
    return {"name": name, **c} if name else c


def listed():
    back = {"op": "route_backward"}
    return [
        # one token of one user: the shortest call there is, all latency
        _route("route_one_token", 1, 256, 8, 8, 16, G=8, top_g=4, rule="top2", scale=2.5),
        # a decode batch of 8 x 128 tokens over 256 experts in 8 groups, biased for balance
        _route("route_decode", 1024, 256, 8, 8, 128, G=8, top_g=4, rule="top2", scale=2.5),
        # softmax scores that are not renormalised, 160 experts in 8 groups ranked by their best, a ragged batch
        _route("route_softmax_groups", 3001, 160, 6, 8, 256, score="softmax", bias=False, G=8, top_g=3,
               renorm=False, scale=16.0),
        # a long prefill with bf16 logits (many ties) that overflows some experts' capacity
        _route("route_prefill_bf16", 16384, 256, 8, 8, 544, G=8, top_g=4, rule="top2", scale=2.5, logits="bf16"),
        # a training micro-batch: the gradient reaches the chosen experts' logits only
        {**_route("route_backward_sigmoid", 4096, 256, 8, 8, 1024, G=8, top_g=4, rule="top2", scale=2.5), **back},
        # softmax over all experts, not renormalised: every logit has a gradient; bf16 logits, odd batch
        {**_route("route_backward_softmax", 32749, 64, 6, 4, 4096, score="softmax", bias=False, renorm=False,
                  logits="bf16"), **back},
        # a small ragged batch with overflowing experts
        _combine("combine_backward_ragged", 237, 2056, 64, 6, 24),
        # a training micro-batch of 8 experts, top-2
        _combine("combine_backward_top2", 4096, 4096, 8, 2, 2048),
        # a training micro-batch of 256 experts, top-8
        _combine("combine_backward_top8", 4096, 7168, 256, 8, 256),
        # one token through the gate and up matrices of its 8 experts: every weight is read for one row
        _w4("expert_w4_one_token", 1, 256, 8, 8, 7168, 2048, act="silu"),
        # fp8 rows, small groups, sizes that no tile divides: a few rows for each of 64 experts
        _w4("expert_w4_ragged_fp8", 77, 64, 6, 24, 1408, 2056, group=32, x="fp8"),
        # the decode batch of 1024 tokens: 32 rows for each of 256 experts
        _w4("expert_w4_decode", 1024, 256, 8, 64, 7168, 2048, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "expert_w4"])
    if op in ("route", "route_backward"):
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * rng.choice([n for n in (4, 7, 8, 16, 20, 32, 40, 64, 128, 256) if 8 <= n * G <= 512])
        top_g = rng.randint(1, G)
        k = rng.randint(1, min(16, top_g * (E // G)))
        T = _log(rng, 1, min(16384, 16384 * 256 // E))
        score, bias = rng.choice([("softmax", False), ("sigmoid", False), ("sigmoid", True)])
        return {**_route(None, T, E, k, G, max(1, int(T * k / E * rng.uniform(0.7, 2.0))), score, bias, G, top_g,
                         rng.choice(["max", "top2"]), rng.random() < 0.6, rng.choice([1.0, 2.5, 16.0]),
                         rng.choice(["f32", "bf16"])), "op": op}
    if op == "combine_backward":
        E = rng.choice([4, 8, 20, 64, 160, 256])
        k = rng.randint(1, min(8, E))
        H = 8 * _log(rng, 16, 896)
        T = _log(rng, 1, max(2, int(4096 * 8 * 7168 / (k * H) / 2)))
        T = min(T, 8192)
        return _combine(None, T, H + 8 * (H == 3072), E, k, max(1, int(T * k / E * rng.uniform(0.7, 2.0))))
    x = rng.choice(["bf16", "bf16", "fp8"])
    group = rng.choice([32, 64, 128])
    n_in = 128 * round(_log(rng, 256, 7168) / 128)
    n_in += 128 * (n_in == 3072)
    n_out = 8 * _log(rng, 32, 512)
    n_out += 8 * (n_out == 3072)
    E = rng.choice([1, 8, 20, 64, 128])
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, max(2, min(1024, 48 * E // k)))
    return _w4(None, T, E, k, max(1, min(T, int(T * k / E * 2) + 4)), n_in, n_out, group,
               rng.choice(["none", "silu"]), x)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _slots(idx, E, C):
    """Slot of every (token, choice) pair: how many earlier tokens chose the same expert, or -1 from C on; counts."""
    T = idx.shape[0]
    hot = torch.zeros((T, E), dtype=torch.int32, device=idx.device)
    hot.scatter_(1, idx, 1)
    before = hot.cumsum(0, dtype=torch.int32) - hot
    slot = before.gather(1, idx)
    return torch.where(slot < C, slot, -1).to(torch.int32), hot.sum(0, dtype=torch.int32)


def _gate_inputs(case, g):
    T, E = case["T"], case["E"]
    l = torch.randn((T, E), device=DEV, generator=g)
    bias = 0.1 * torch.randn(E, device=DEV, generator=g) if case["bias"] else None
    return (l.to(torch.bfloat16) if case["logits"] == "bf16" else l), bias


def _random_routing(T, E, k, C, g):
    """k distinct experts for each token, their softmax weights and slots."""
    l = torch.randn((T, E), device=DEV, generator=g)
    top, idx = l.topk(k, dim=1)
    slot, counts = _slots(idx, E, C)
    return idx.to(torch.int32), torch.softmax(top, 1), slot, counts


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, T, E, k, C = case["op"], case["T"], case["E"], case["k"], case["C"]
    st = {"case": case}
    if op in ("route", "route_backward"):
        st["logits"], st["bias"] = _gate_inputs(case, g)
        i32 = {"dtype": torch.int32, "device": DEV}
        if op == "route":
            st["out"] = {"topk_idx": torch.empty((T, k), **i32), "topk_w": torch.empty((T, k), device=DEV),
                         "counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
                         "slot": torch.empty((T, k), **i32), "rank_counts": torch.empty(case["R"], **i32),
                         "dropped": torch.empty(1, **i32)}
        else:
            idx, w = _gate(case, st["logits"], st["bias"])
            st["idx"], st["w"] = idx.to(torch.int32), w
            st["d_w"] = torch.randn((T, k), device=DEV, generator=g)
            st["d_logits"] = torch.empty_like(st["logits"])
    elif op == "combine_backward":
        H = case["H"]
        st["idx"], st["w"], st["slot"], _ = _random_routing(T, E, k, C, g)
        st["y"] = torch.randn((E, C, H), device=DEV, generator=g, dtype=torch.bfloat16)
        st["d_out"] = torch.randn((T, H), device=DEV, generator=g, dtype=torch.bfloat16)
        st["d_y"] = torch.zeros((E, C, H), dtype=torch.bfloat16, device=DEV)     # rows of no pair stay as they are
        st["d_w"] = torch.empty((T, k), device=DEV)
    else:
        K, N, grp = case["n_in"], case["n_out"], case["group"]
        rows = 2 * N if case["act"] == "silu" else N
        _, _, _, st["counts"] = _random_routing(T, E, k, C, g)
        x = torch.randn((E, C, K), device=DEV, generator=g, dtype=torch.bfloat16)
        st["x_scale"] = None
        if case["x"] == "fp8":
            b = x.float().unflatten(-1, (-1, 128))
            s = b.abs().amax(-1) / 448.0
            st["x_scale"] = s
            x = (b / s[..., None]).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
        st["x"] = x
        # every byte holds two codes, so uniform bytes are packed uniform codes
        st["w_q"] = torch.randint(0, 256, (E, rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)
        st["w_scale"] = ((1.0 + torch.rand((E, rows, K // grp), device=DEV, generator=g)) *
                         (0.15 / math.sqrt(K))).to(torch.bfloat16)
        st["y"] = torch.zeros((E, C, N), dtype=torch.bfloat16, device=DEV)       # rows past the counts stay as they are
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _handles(st)
    return st


def _handles(st):
    """The descriptors and workspaces that a program makes once for its sizes."""
    import combine_router_top_gb300 as M
    c = st["case"]
    if c["op"] in ("route", "route_backward"):
        st["p"] = M.problem(c["T"], 8, c["E"], c["k"], c["R"], c["C"])
        st["gate"] = M.gate(score=M.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else M.MOE_SCORE_SOFTMAX,
                            groups=c["G"], top_groups=c["top_g"],
                            group_rule=M.MOE_GROUP_TOP2 if c["rule"] == "top2" else M.MOE_GROUP_MAX,
                            renormalise=c["renorm"], scale=c["scale"],
                            logits_type=M.MOE_LOGITS_BF16 if c["logits"] == "bf16" else M.MOE_LOGITS_F32)
        if c["op"] == "route":
            st["ws"] = torch.empty(M.moe_route_workspace_bytes(st["p"]), dtype=torch.uint8, device=DEV)
    elif c["op"] == "combine_backward":
        st["p"] = M.problem(c["T"], c["H"], c["E"], c["k"], 1, c["C"])
    else:
        dt = M.MOE_DTYPE_FP8_E4M3_B128 if c["x"] == "fp8" else M.MOE_DTYPE_BF16
        st["p"] = M.problem(c["T"], c["n_in"], c["E"], c["k"], 1, c["C"], dt)
        st["w4"] = M.w4(c["n_in"], c["n_out"], group=c["group"],
                        act=M.MOE_ACT_SILU_GATE if c["act"] == "silu" else M.MOE_ACT_NONE)
        st["ws"] = torch.empty(M.moe_expert_w4_workspace_bytes(st["p"], st["w4"]), dtype=torch.uint8, device=DEV)


# ---- plain forms ----------------------------------------------------------------------------------------------------

def _best(key, k):
    """Places of the k largest of each row, largest first, ties to the lowest place."""
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :k]


def _gate(case, logits, bias):
    """Chosen experts and their weights."""
    k, G = case["k"], case["G"]
    l = logits.float()
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(1, keepdim=True))           # softmax times its denominator, which orders alike
    key = s + bias if bias is not None else l                # what the choice goes by
    if G > 1:
        if case["rule"] == "top2":
            two = torch.sort((s + bias if bias is not None else s).unflatten(1, (G, -1)), dim=-1).values[..., -2:]
            best = two.sum(-1)
        else:
            best = key.unflatten(1, (G, -1)).amax(-1)
        live = torch.zeros_like(best, dtype=torch.bool).scatter_(1, _best(best, case["top_g"]), True)
        key = torch.where(live.repeat_interleave(key.shape[1] // G, 1), key, -math.inf)
    idx = _best(key, k)
    if case["renorm"]:
        top = s.gather(1, idx) if case["score"] == "sigmoid" else l.gather(1, idx)
        if case["score"] == "softmax":
            top = torch.exp(top - top.amax(1, keepdim=True))
        w = top / top.sum(1, keepdim=True)
    else:
        w = s.gather(1, idx)
        if case["score"] == "softmax":
            w = w / s.sum(1, keepdim=True)
    return idx, w * case["scale"]


def _plain_route(st):
    c = st["case"]
    idx, w = _gate(c, st["logits"], st["bias"])
    slot, counts = _slots(idx, c["E"], c["C"])
    offsets = torch.nn.functional.pad(counts.cumsum(0, dtype=torch.int32), (1, 0))
    kept = counts.clamp(max=c["C"])
    return {"topk_idx": idx.to(torch.int32), "topk_w": w, "counts": counts, "offsets": offsets, "slot": slot,
            "rank_counts": kept.view(c["R"], -1).sum(1, dtype=torch.int32),
            "dropped": (counts - kept).sum(0, keepdim=True, dtype=torch.int32)}


def _plain_route_backward(st):
    c = st["case"]
    l, idx, w, d_w = st["logits"].float(), st["idx"].long(), st["w"], st["d_w"]
    dot = (w * d_w).sum(1, keepdim=True) / c["scale"]
    if c["score"] == "softmax" and not c["renorm"]:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        d = torch.zeros_like(l).scatter_(1, idx, d_w)
        return (c["scale"] * p * (d - dot)).to(st["logits"].dtype)
    d = w * (d_w - dot) if c["renorm"] else w * d_w
    if c["score"] == "sigmoid":
        d = d / (1.0 + torch.exp(l.gather(1, idx)))          # times 1 - sigmoid
    return torch.zeros_like(l).scatter_(1, idx, d).to(st["logits"].dtype)


def _plain_combine_backward(st):
    idx, slot, C = st["idx"].long(), st["slot"].long(), st["case"]["C"]
    kept = slot >= 0
    rows = (idx * C + slot)[kept]                            # each row of a pair is that pair's alone
    token = torch.nonzero(kept)[:, 0]
    d_out = st["d_out"].float()[token]
    st["d_y"].view(-1, st["case"]["H"])[rows] = (st["w"][kept][:, None] * d_out).to(torch.bfloat16)
    d_w = torch.zeros_like(st["w"])
    d_w[kept] = (st["y"].view(-1, st["case"]["H"])[rows].float() * d_out).sum(1)
    return {"d_y": st["d_y"], "d_topk_w": d_w}


def _unpack(q):
    """Codes 0..15 of packed rows [..., K/2], in the inputs' order. A row holds blocks of 128 inputs, 64 bytes each;
    the little-endian 32-bit word 4 t + j of a block (t, j < 4) holds its inputs 32 j + 8 t .. 32 j + 8 t + 7, the
    even ones' codes in the low 16 bits and the odd ones' in the high 16."""
    b = q.unflatten(-1, (-1, 4, 4, 4))                       # block, t, j, byte
    lo, hi = b & 15, b >> 4
    word = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1],
                        hi[..., 3]], -1)                     # block, t, j, input of the word
    return word.transpose(-2, -3).flatten(-4)


def _plain_expert_w4(st):
    c = st["case"]
    E, C, K, N, grp = c["E"], c["C"], c["n_in"], c["n_out"], c["group"]
    e = torch.nonzero(st["counts"])[:, 0]                    # the experts that have rows
    w = (_unpack(st["w_q"][e]).float() - 8.0).unflatten(-1, (-1, grp)) * st["w_scale"][e].float()[..., None]
    x = st["x"][e]
    if c["x"] == "fp8":
        x = (x.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)) * st["x_scale"][e][..., None]).flatten(-2)
    r = torch.bmm(x.float(), w.flatten(-2).transpose(1, 2))
    if c["act"] == "silu":
        gate, up = r[..., :N], r[..., N:]
        r = gate / (1.0 + torch.exp(-gate)) * up
    live = torch.arange(C, device=r.device)[None, :, None] < st["counts"][e][:, None, None]
    st["y"][e] = torch.where(live, r.to(torch.bfloat16), st["y"][e])
    return st["y"]


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if not own:
        if op == "route":
            return _plain_route(st)
        if op == "route_backward":
            return _plain_route_backward(st)
        if op == "combine_backward":
            return _plain_combine_backward(st)
        return _plain_expert_w4(st)
    import combine_router_top_gb300 as M
    if op == "route":
        o = st["out"]
        M.moe_route_gated(st["p"], st["gate"], st["logits"], st["bias"], o["topk_idx"], o["topk_w"], o["counts"],
                          o["offsets"], o["slot"], o["rank_counts"], o["dropped"], st["ws"])
        return o
    if op == "route_backward":
        M.moe_route_gated_backward(st["p"], st["gate"], st["logits"], st["idx"], st["w"], st["d_w"], st["d_logits"])
        return st["d_logits"]
    if op == "combine_backward":
        M.moe_combine_backward(st["p"], st["y"], st["d_out"], st["idx"], st["w"], st["slot"], st["d_y"], st["d_w"])
        return {"d_y": st["d_y"], "d_topk_w": st["d_w"]}
    M.moe_expert_w4(st["p"], st["w4"], st["x"], st["x_scale"], st["counts"], st["w_q"], st["w_scale"], st["y"],
                    st["ws"])
    return st["y"]


def work(case):
    op, T, E, k, C = case["op"], case["T"], case["E"], case["k"], case["C"]
    if op in ("route", "route_backward"):
        size = 2 if case["logits"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * E * size + 4 * E * case["bias"] + T * k * 12 + (2 * E + case["R"] + 2) * 4,
                    "flops": 4 * T * E}
        dense = case["score"] == "softmax" and not case["renorm"]
        # the logits that the formula needs: all, the chosen ones (sigmoid), or none (the weights say it)
        read = T * E if dense else T * k if case["score"] == "sigmoid" else 0
        return {"bytes": read * size + T * E * size + T * k * 12, "flops": (8 * T * E if dense else 0) + 8 * T * k}
    kept = min(T * k, E * C)
    if op == "combine_backward":
        H = case["H"]
        return {"bytes": 2 * kept * H * 2 + T * H * 2 + T * k * 16, "flops": 3 * kept * H}
    K, N = case["n_in"], case["n_out"]
    rows = 2 * N if case["act"] == "silu" else N
    live = E * (1.0 - (1.0 - k / E) ** T)                    # experts that some token chose
    x = K + K // 32 if case["x"] == "fp8" else 2 * K
    return {"bytes": live * rows * (K / 2 + K / case["group"] * 2) + kept * (x + 2 * N) + 4 * E,
            "flops": 2.0 * kept * rows * K}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def _choice64(case, logits, bias):
    """Chosen experts, their scores before renormalisation and all scores, in 64 bits."""
    l = logits.double()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    key = s if bias is None else s + bias.double()
    per = case["E"] // case["G"]
    if case["G"] > 1:
        by = key.view(-1, case["G"], per).topk(2 if case["rule"] == "top2" else 1, dim=2).values.sum(2)
        keep = torch.zeros_like(by).scatter_(1, _best(by, case["top_g"]), 1.0).repeat_interleave(per, 1)
        key = key.masked_fill(keep == 0, -math.inf)
    idx = _best(key, case["k"])
    return idx, s.gather(1, idx), s


def exact(case, seed):
    st = _inputs(case, seed)
    op, C = case["op"], case["C"]
    if op == "route":
        # whole numbers have no rounding: the choice, and what is counted from it, is compared as it is
        _, s, _ = _choice64(case, st["logits"], st["bias"])
        w = (s / s.sum(1, keepdim=True) if case["renorm"] else s) * case["scale"]
        return {"topk_idx": None, "topk_w": w, "counts": None, "offsets": None, "slot": None, "rank_counts": None,
                "dropped": None}
    if op == "route_backward":
        l, idx, d_w = st["logits"].double(), st["idx"].long(), st["d_w"].double()
        l.requires_grad_(True)
        s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        w = s.gather(1, idx)
        w = (w / w.sum(1, keepdim=True) if case["renorm"] else w) * case["scale"]
        return torch.autograd.grad(w, l, d_w)[0]
    if op == "combine_backward":
        T, k, H = case["T"], case["k"], case["H"]
        y, w = st["y"].double(), st["w"].double()
        d_y, d_w = torch.zeros_like(y), torch.zeros((T, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            t = torch.nonzero(st["slot"][:, j] >= 0)[:, 0]
            e, s = st["idx"][t, j].long(), st["slot"][t, j].long()
            d_y[e, s] = w[t, j, None] * st["d_out"][t].double()
            d_w[t, j] = (y[e, s] * st["d_out"][t].double()).sum(1)
        return {"d_y": d_y, "d_topk_w": d_w}
    y = st["y"].double()
    for e, n in enumerate(st["counts"].clamp(max=C).tolist()):
        if n == 0:
            continue
        i = torch.arange(case["n_in"], device=DEV)                          # where input i's code stands
        word = i // 128 * 16 + i % 32 // 8 * 4 + i % 128 // 32
        q = (st["w_q"][e].view(torch.int32)[:, word] >> (i % 8 // 2 * 4 + i % 2 * 16).int() & 15).double() - 8
        w = q * st["w_scale"][e].double().repeat_interleave(case["group"], 1)
        x = st["x"][e, :n]
        x = x.double() if case["x"] == "bf16" else \
            x.view(torch.float8_e4m3fn).double() * st["x_scale"][e, :n].double().repeat_interleave(128, 1)
        r = x @ w.T
        if case["act"] == "silu":
            r = torch.nn.functional.silu(r[:, :case["n_out"]]) * r[:, case["n_out"]:]
        y[e, :n] = r
    return y
