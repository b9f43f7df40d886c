"""Performance cases of the norms around a mixture-of-experts block and of the whole layer for a few tokens.

    block_norm           moe_block_norm: the norm after a block, its gate and residual scale, the sum with the residual
                         stream and the norm before the next block
    combine_norm         moe_combine_norm: the same behind the weighted sum of the experts' rows, which is formed on
                         the way
    block_norm_backward  moe_block_norm_backward: the gradients of the block's output, the residual stream, both norms'
                         weights and the gate
    layer_few            moe_layer_few: choice, gate and up products, SiLU, down product and weighted sum for up to 32
                         tokens, with bf16, e4m3 or 4-bit weights and, where asked for, an expert that every token shares

Each case is run in a plain form (elementary torch operations in 32 bits, rounded once at the end) or, where `own` is
set, by the calls of the package.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------------------------------

def _norm(op, name, T, H, gate="none", res="bf16", par="bf16", scale=1.0, post=True, **more):
    c = {"op": op, "T": T, "H": H, "gate": gate, "res": res, "par": par, "scale": scale, "post": post, **more}
    return {"name": name, **c} if name else c


def _few(name, T, E, k, H, inner, weights="bf16", group=128, shared=0, score="sigmoid", G=1, top_g=1, scale=1.0):
    c = {"op": "layer_few", "T": T, "E": E, "k": k, "H": H, "inner": inner, "weights": weights, "group": group,
         "shared": shared, "score": score, "G": G, "top_g": top_g, "scale": scale}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of one user: the shortest call, all latency
        _norm("block_norm", "block_norm_one_token", 1, 7168),
        # fp32 residual stream, fp32 weights, a gate for each token, sizes that no tile divides
        _norm("block_norm", "block_norm_ragged_f32", 3001, 2056, gate="token", res="f32", par="f32", scale=0.5),
        # a long prefill: norms before and after the block
        _norm("block_norm", "block_norm_prefill", 16384, 7168),
        # the decode batch of 1024 tokens over 256 experts: 8 rows to a token
        _norm("combine_norm", "combine_norm_decode", 1024, 7168, E=256, k=8, C=128, keep=False),
        # a small training batch with overflowing experts; the combine's output is kept for the way back
        _norm("combine_norm", "combine_norm_ragged", 237, 2056, gate="channel", res="f32", E=64, k=6, C=24, keep=True),
        # small and ragged, a gate for each token
        _norm("block_norm_backward", "backward_ragged", 237, 2056, gate="token", res="f32", par="f32", scale=0.5),
        # a training micro-batch with a gate for each channel
        _norm("block_norm_backward", "backward_micro_batch", 4096, 7168, gate="channel"),
        # a long training batch, odd, without a norm after the block
        _norm("block_norm_backward", "backward_long", 16381, 4096, post=False),
        # one token, 8 of 256 experts and the shared one, 4-bit weights: latency counts
        _few("few_one_token_w4", 1, 256, 8, 7168, 2048, "w4", shared=1, G=8, top_g=4, scale=2.5),
        # one token, 2 of 8 large experts, bf16 weights
        _few("few_one_token_bf16", 1, 8, 2, 4096, 14336, score="softmax"),
        # a few users' tokens, many small experts and a shared one, fp8 weights
        _few("few_ragged_fp8", 13, 64, 6, 2048, 1408, "fp8", shared=1, score="softmax"),
        # the most tokens there are, spread over 256 experts, fp8 weights
        _few("few_batch_fp8", 32, 256, 8, 7168, 2048, "fp8", G=8, top_g=4, scale=2.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_norm", "combine_norm", "block_norm_backward", "layer_few", "layer_few"])
    if op == "layer_few":
        weights = rng.choice(["bf16", "fp8", "w4"])
        E = rng.choice([4, 8, 20, 64, 160, 256])
        step = 64 if weights == "bf16" else 128
        H = step * max(1, round(_log(rng, 256, 7168) / step))
        per = int(1.5e9 / (E * 3 * H * {"bf16": 2, "fp8": 1, "w4": 0.5}[weights]))
        inner = step * max(1, round(_log(rng, 128, max(129, min(8192, per))) / step))
        G = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        top_g = rng.randint(1, G)
        k = rng.randint(1, min(8, top_g * (E // G)))
        return _few(None, _log(rng, 1, 32), E, k, H, inner, weights, rng.choice([32, 64, 128]), rng.randint(0, 1),
                    rng.choice(["softmax", "sigmoid"]), G, top_g, rng.choice([1.0, 2.5]))
    H = 8 * _log(rng, 16, 2048)
    more = {}
    cap = 16384 * 7168
    if op == "combine_norm":
        E = rng.choice([4, 8, 20, 64, 160, 256])
        k = rng.randint(1, min(8, E))
        cap = 1024 * 7168 * 8 // k
    T = _log(rng, 1, max(2, min(32768, cap // H // (2 if op == "block_norm_backward" else 1))))
    if op == "combine_norm":
        more = {"E": E, "k": k, "C": max(1, int(T * k / E * rng.uniform(0.7, 2.0))), "keep": rng.random() < 0.5}
    return _norm(op, None, T, H, rng.choice(["none", "channel", "token"]), rng.choice(["bf16", "bf16", "f32"]),
                 rng.choice(["bf16", "f32"]), rng.choice([1.0, 0.5, 0.22]), rng.random() < 0.7, **more)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _slots(idx, E, C):
    """Slot of every (token, choice) pair: how many earlier tokens chose the same expert, or -1 from C on."""
    hot = torch.zeros((idx.shape[0], E), dtype=torch.int32, device=idx.device)
    hot.scatter_(1, idx, 1)
    slot = (hot.cumsum(0, dtype=torch.int32) - hot).gather(1, idx)
    return torch.where(slot < C, slot, -1).to(torch.int32)


def _matrices(c, g, rows, cols):
    """One matrix [rows][cols] for each expert, entries of about cols ** -0.5, and its scales."""
    n = c["E"] + c["shared"]
    if c["weights"] == "w4":
        # every byte holds two codes, so uniform bytes are packed uniform codes
        q = torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device=DEV, generator=g)
        s = (1.0 + torch.rand((n, rows, cols // c["group"]), device=DEV, generator=g)) * (0.15 / math.sqrt(cols))
        return q, s.to(torch.bfloat16)
    if c["weights"] == "bf16":
        w = torch.empty((n, rows, cols), dtype=torch.bfloat16, device=DEV)
        for e in range(n):
            w[e].normal_(0.0, 1.0 / math.sqrt(cols), generator=g)
        return w, None
    q = torch.empty((n, rows, cols), dtype=torch.uint8, device=DEV)
    for e in range(n):
        v = 64.0 * torch.randn((rows, cols), dtype=torch.bfloat16, device=DEV, generator=g)
        q[e] = v.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s = (1.0 + torch.rand((n, rows // 128, cols // 128), device=DEV, generator=g)) * (0.0107 / math.sqrt(cols))
    return q, s


def _inputs(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    T, H, op = c["T"], c["H"], c["op"]

    def rows(*shape, dtype=torch.bfloat16, scale=1.0):
        return (scale * torch.randn(shape, device=DEV, generator=g)).to(dtype)
    st = {"case": case}
    if op == "layer_few":
        E, k = c["E"], c["k"]
        st["x"], st["logits"] = rows(T, H), rows(T, E, dtype=torch.float32)
        st["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g) if c["score"] == "sigmoid" else None
        st["w_up"], st["up_scale"] = _matrices(c, g, 2 * c["inner"], H)
        st["w_down"], st["down_scale"] = _matrices(c, g, H, c["inner"])
        st["topk_idx"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        st["topk_w"] = torch.empty((T, k), device=DEV)
        st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        return st
    res, par = _type(c["res"]), _type(c["par"])
    if op == "combine_norm":
        E, k, C = c["E"], c["k"], c["C"]
        top, idx = torch.randn((T, E), device=DEV, generator=g).topk(k, dim=1)
        st["idx"], st["w"], st["slot"] = idx.to(torch.int32), torch.softmax(top, 1), _slots(idx, E, C)
        st["y"] = torch.randn((E, C, H), device=DEV, generator=g, dtype=torch.bfloat16)
        st["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV) if c["keep"] else None
    else:
        st["y"] = rows(T, H)
    st["w_post"] = (1.0 + 0.1 * torch.randn(H, device=DEV, generator=g)).to(par) if c["post"] else None
    st["w_pre"] = (1.0 + 0.1 * torch.randn(H, device=DEV, generator=g)).to(par)
    st["gate"] = (0.3 * torch.randn(H, device=DEV, generator=g)).to(par) if c["gate"] == "channel" else \
        torch.rand(T, device=DEV, generator=g) if c["gate"] == "token" else None
    if op == "block_norm_backward":
        # a residual stream grows over the layers, and some of its channels far above the others
        st["r"] = (rows(T, H, dtype=torch.float32, scale=2.0) *
                   (1.0 + 9.0 * (torch.rand(H, device=DEV, generator=g) < 0.01))).to(res)
        st["d_r"], st["d_n"] = rows(T, H, dtype=res), rows(T, H)
        st["d_y"], st["d_residual"] = torch.empty_like(st["y"]), torch.empty_like(st["r"])
        f32 = {"dtype": torch.float32, "device": DEV}
        st["d_w_post"] = torch.empty(H, **f32) if c["post"] else None
        st["d_w_pre"] = torch.empty(H, **f32)
        st["d_gate"] = torch.empty(H if c["gate"] == "channel" else T, **f32) if c["gate"] != "none" else None
    else:
        st["residual"] = (rows(T, H, dtype=torch.float32, scale=2.0) *
                          (1.0 + 9.0 * (torch.rand(H, device=DEV, generator=g) < 0.01))).to(res)
        st["r"], st["n"] = torch.empty_like(st["residual"]), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
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
    if c["op"] == "layer_few":
        st["p"] = M.problem(c["T"], c["H"], c["E"], c["k"], 1, c["T"])
        st["how"] = M.gate(score=M.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else M.MOE_SCORE_SOFTMAX,
                           groups=c["G"], top_groups=c["top_g"],
                           group_rule=M.MOE_GROUP_TOP2 if c["score"] == "sigmoid" else M.MOE_GROUP_MAX,
                           scale=c["scale"])
        st["mlp"] = M.mlp(c["inner"], {"bf16": M.MOE_WEIGHTS_BF16, "fp8": M.MOE_WEIGHTS_FP8_B128,
                                       "w4": M.MOE_WEIGHTS_W4}[c["weights"]], group=c["group"], shared=c["shared"])
        n = M.moe_layer_few_workspace_bytes(st["p"], st["mlp"])
    else:
        E, k, C = (c["E"], c["k"], c["C"]) if c["op"] == "combine_norm" else (1, 1, 1)
        st["p"] = M.problem(c["T"], c["H"], E, k, 1, C)
        st["norm"] = M.norm(eps=EPS, scale=c["scale"], residual=M.MOE_VALUE_F32 if c["res"] == "f32" else M.MOE_VALUE_BF16,
                            params=M.MOE_VALUE_F32 if c["par"] == "f32" else M.MOE_VALUE_BF16,
                            gate={"none": M.MOE_BRANCH_PLAIN, "channel": M.MOE_BRANCH_CHANNEL,
                                  "token": M.MOE_BRANCH_TOKEN}[c["gate"]])
        n = M.moe_block_norm_backward_workspace_bytes(st["p"], st["norm"]) if c["op"] == "block_norm_backward" else 0
    st["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)


# ---- plain forms ----------------------------------------------------------------------------------------------------

def _rms(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _gate_of(st):
    """The branch's factor a g, as it broadcasts over the rows."""
    c, g = st["case"], st["gate"]
    if g is None:
        return c["scale"]
    return c["scale"] * (g.float()[:, None] if c["gate"] == "token" else g.float())


def _join(st, y):
    b = y if st["w_post"] is None else y * _rms(y) * st["w_post"].float()
    r = st["residual"].float() + _gate_of(st) * b
    n = r * _rms(r) * st["w_pre"].float()
    return {"r": r.to(st["residual"].dtype), "n": n.to(torch.bfloat16)}


def _plain_combine_norm(st):
    c = st["case"]
    rows = st["y"].view(-1, c["H"])
    y = torch.zeros((c["T"], c["H"]), device=DEV)
    for j in range(c["k"]):
        s = st["slot"][:, j]
        row = st["idx"][:, j] * c["C"] + s.clamp(min=0)
        y += torch.where(s[:, None] >= 0, st["w"][:, j, None] * rows[row.long()].float(), 0.0)
    out = _join(st, y)
    return {"out": y.to(torch.bfloat16), **out} if c["keep"] else out


def _plain_backward(st):
    c = st["case"]
    y, r, d_n, w_pre = st["y"].float(), st["r"].float(), st["d_n"].float(), st["w_pre"].float()
    rs = _rms(r)
    rh = r * rs
    v = w_pre * d_n
    D = st["d_r"].float() + rs * (v - rh * (rh * v).mean(1, keepdim=True))
    out = {"d_residual": D.to(st["r"].dtype), "d_w_pre": (d_n * rh).sum(0)}
    f = _gate_of(st) * D                                     # the gradient of what the gate multiplies
    b = y
    if c["post"]:
        ys = _rms(y)
        yh = y * ys
        b = yh * st["w_post"].float()
        v = st["w_post"].float() * f
        out["d_y"] = (ys * (v - yh * (yh * v).mean(1, keepdim=True))).to(torch.bfloat16)
        out["d_w_post"] = (f * yh).sum(0)
    else:
        out["d_y"] = f.to(torch.bfloat16)
    if c["gate"] != "none":
        out["d_gate"] = c["scale"] * (D * b).sum(1 if c["gate"] == "token" else 0)
    return out


def _best(key, k):
    """Places of the k largest of each row, largest first, ties to the lowest place."""
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :k]


def _choose(st):
    c, l = st["case"], st["logits"]
    k, G = c["k"], c["G"]
    sig = c["score"] == "sigmoid"
    s = 1.0 / (1.0 + torch.exp(-l)) if sig else torch.exp(l - l.amax(1, keepdim=True))
    key = s + st["bias"] if sig else l
    if G > 1:
        groups = torch.sort(key.unflatten(1, (G, -1)), dim=-1).values[..., -2 if sig else -1:].sum(-1)
        live = torch.zeros_like(groups, dtype=torch.bool).scatter_(1, _best(groups, c["top_g"]), True)
        key = torch.where(live.repeat_interleave(c["E"] // G, 1), key, -math.inf)
    idx = _best(key, k)
    w = s.gather(1, idx)
    return idx, w / w.sum(1, keepdim=True) * c["scale"]


def _unpack(q):
    """Codes 0..15 of packed rows [..., K/2], in the inputs' order. A row holds blocks of 128 inputs, 64 bytes each;
    the little-endian 32-bit word 4 t + j of a block (t, j < 4) holds its inputs 32 j + 8 t .. 32 j + 8 t + 7, the
    even ones' codes in the low 16 bits and the odd ones' in the high 16."""
    b = q.unflatten(-1, (-1, 4, 4, 4))                       # block, t, j, byte
    lo, hi = b & 15, b >> 4
    word = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1],
                        hi[..., 3]], -1)                     # block, t, j, input of the word
    return word.transpose(-2, -3).flatten(-4)


def _matrix(c, w, scale, e):
    if c["weights"] == "bf16":
        return w[e].float()
    if c["weights"] == "fp8":
        s = scale[e].repeat_interleave(128, 0).repeat_interleave(128, 1)
        return w[e].view(torch.float8_e4m3fn).float() * s
    q = _unpack(w[e]).float() - 8.0
    return (q.unflatten(-1, (-1, c["group"])) * scale[e].float()[..., None]).flatten(-2)


def _plain_few(st):
    c, I = st["case"], st["case"]["inner"]
    idx, w = _choose(st)
    out = torch.zeros((c["T"], c["H"]), device=DEV)
    x = st["x"].float()
    pairs = [(e, None) for e in torch.unique(idx).tolist()]
    if c["shared"]:
        pairs.append((c["E"], slice(None)))
    for e, rows in pairs:
        if rows is None:
            rows, j = torch.nonzero(idx == e, as_tuple=True)
            weight = w[rows, j, None]
        else:
            weight = 1.0
        r = x[rows] @ _matrix(c, st["w_up"], st["up_scale"], e).T
        h = r[:, :I] / (1.0 + torch.exp(-r[:, :I])) * r[:, I:]
        out[rows] += weight * (h @ _matrix(c, st["w_down"], st["down_scale"], e).T)
    return {"topk_idx": idx.to(torch.int32), "topk_w": w, "out": out.to(torch.bfloat16)}


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(st):
    c, op = st["case"], st["case"]["op"]
    if not own:
        if op == "block_norm":
            return _join(st, st["y"].float())
        return {"combine_norm": _plain_combine_norm, "block_norm_backward": _plain_backward,
                "layer_few": _plain_few}[op](st)
    import combine_router_top_gb300 as M
    if op == "block_norm":
        M.moe_block_norm(st["p"], st["norm"], st["y"], st["residual"], st["w_post"], st["w_pre"], st["gate"], st["r"],
                         st["n"])
        return {"r": st["r"], "n": st["n"]}
    if op == "combine_norm":
        M.moe_combine_norm(st["p"], st["norm"], st["y"], st["idx"], st["w"], st["slot"], st["residual"], st["w_post"],
                           st["w_pre"], st["gate"], st["out"], st["r"], st["n"])
        out = {"r": st["r"], "n": st["n"]}
        return {"out": st["out"], **out} if c["keep"] else out
    if op == "block_norm_backward":
        M.moe_block_norm_backward(st["p"], st["norm"], st["y"], st["r"], st["d_r"], st["d_n"], st["w_post"], st["w_pre"],
                                  st["gate"], st["d_y"], st["d_residual"], st["d_w_post"], st["d_w_pre"], st["d_gate"],
                                  st["ws"])
        out = {"d_residual": st["d_residual"], "d_w_pre": st["d_w_pre"], "d_y": st["d_y"]}
        if c["post"]:
            out["d_w_post"] = st["d_w_post"]
        if c["gate"] != "none":
            out["d_gate"] = st["d_gate"]
        return out
    M.moe_layer_few(st["p"], st["how"], st["mlp"], st["x"], st["logits"], st["bias"], st["w_up"], st["up_scale"],
                    st["w_down"], st["down_scale"], st["topk_idx"], st["topk_w"], st["out"], st["ws"])
    return {"topk_idx": st["topk_idx"], "topk_w": st["topk_w"], "out": st["out"]}


def work(case):
    c, T, H = case, case["T"], case["H"]
    if c["op"] == "layer_few":
        E, k, I = c["E"], c["k"], c["inner"]
        live = E * (1.0 - (1.0 - k / E) ** T) + c["shared"]          # experts that some token chose
        per = {"bf16": 2.0, "fp8": 1.0 + 4.0 / 128 ** 2, "w4": 0.5 + 2.0 / c["group"]}[c["weights"]]
        return {"bytes": live * 3 * H * I * per + T * (4 * H + 4 * E + 8 * k),
                "flops": 2.0 * T * (k + c["shared"]) * 3 * H * I}
    res, par = (4 if c["res"] == "f32" else 2), (4 if c["par"] == "f32" else 2)
    side = H * par * (1 + c["post"] + (c["gate"] == "channel")) + 4 * T * (c["gate"] == "token")
    if c["op"] == "block_norm":
        return {"bytes": T * H * (4 + 2 * res) + side, "flops": 10 * T * H}
    if c["op"] == "combine_norm":
        kept = min(T * c["k"], c["E"] * c["C"])
        return {"bytes": kept * H * 2 + T * c["k"] * 12 + T * H * (2 + 2 * res + 2 * c["keep"]) + side,
                "flops": 2 * kept * H + 10 * T * H}
    return {"bytes": T * H * (6 + 3 * res) + side + 4 * H * (1 + c["post"] + (c["gate"] == "channel")) +
            4 * T * (c["gate"] == "token"), "flops": 30 * T * H}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------

def _norm64(v, w):
    v = v / (v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt()
    return v if w is None else v * w.double()


def _branch64(st, y, w_post, gate):
    c = st["case"]
    b = _norm64(y, w_post) if w_post is not None else y
    if gate is not None:
        b = b * (gate.unsqueeze(1) if c["gate"] == "token" else gate)
    return c["scale"] * b


def _exact_backward(st):
    c = st["case"]
    leaf = {n: st[n].double().requires_grad_(True) for n in ("y", "r", "w_pre")}
    for n in ("w_post", "gate"):
        leaf[n] = st[n].double().requires_grad_(True) if st[n] is not None else None
    n = _norm64(leaf["r"], leaf["w_pre"])
    through, d_w_pre = torch.autograd.grad(n, [leaf["r"], leaf["w_pre"]], st["d_n"].double())
    D = st["d_r"].double() + through
    wanted = [m for m in ("y", "w_post", "gate") if leaf[m] is not None]
    got = torch.autograd.grad(_branch64(st, leaf["y"], leaf["w_post"], leaf["gate"]), [leaf[m] for m in wanted], D)
    return {"d_residual": D, "d_w_pre": d_w_pre, **{"d_" + m: v for m, v in zip(wanted, got)}}


def _matrix64(c, w, scale, e):
    if c["weights"] == "bf16":
        return w[e].double()
    if c["weights"] == "fp8":
        v = w[e].view(torch.float8_e4m3fn).double()
        n, m = v.shape
        return (v.view(n // 128, 128, m // 128, 128) * scale[e].double()[:, None, :, None]).view(n, m)
    i = torch.arange(2 * w.shape[-1], device=DEV)                    # where input i's code stands
    word = i // 128 * 16 + i % 32 // 8 * 4 + i % 128 // 32
    q = (w[e].view(torch.int32)[:, word] >> (i % 8 // 2 * 4 + i % 2 * 16).int() & 15).double() - 8
    return q * scale[e].double().repeat_interleave(c["group"], 1)


def _exact_few(st):
    c, k, G = st["case"], st["case"]["k"], st["case"]["G"]
    l, sig = st["logits"].double(), st["case"]["score"] == "sigmoid"
    s = torch.sigmoid(l) if sig else torch.softmax(l, 1)
    key = s + st["bias"].double() if sig else s
    if G > 1:
        by = key.view(-1, G, c["E"] // G).topk(2 if sig else 1, dim=2).values.sum(2)
        keep = torch.zeros_like(by).scatter_(1, _best(by, c["top_g"]), 1.0).repeat_interleave(c["E"] // G, 1)
        key = key.masked_fill(keep == 0, -math.inf)
    idx = _best(key, k)
    w = s.gather(1, idx)
    w = w / w.sum(1, keepdim=True) * c["scale"]
    full = torch.zeros((c["T"], c["E"] + c["shared"]), dtype=torch.float64, device=DEV).scatter_(1, idx, w)
    if c["shared"]:
        full[:, -1] = 1.0
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
    for e in torch.nonzero((full != 0).any(0))[:, 0].tolist():
        t = torch.nonzero(full[:, e])[:, 0]
        up = st["x"][t].double() @ _matrix64(c, st["w_up"], st["up_scale"], e).T
        h = torch.nn.functional.silu(up[:, :c["inner"]]) * up[:, c["inner"]:]
        out[t] += full[t, e, None] * (h @ _matrix64(c, st["w_down"], st["down_scale"], e).T)
    return {"topk_idx": None, "topk_w": w, "out": out}


def exact(case, seed):
    st = _inputs(case, seed)
    c, op = case, case["op"]
    if op == "layer_few":
        return _exact_few(st)
    if op == "block_norm_backward":
        return _exact_backward(st)
    y = st["y"].double()
    if op == "combine_norm":
        rows, y = y, torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            t = torch.nonzero(st["slot"][:, j] >= 0)[:, 0]
            y[t] += st["w"][t, j, None].double() * rows[st["idx"][t, j].long(), st["slot"][t, j].long()]
    gate = st["gate"].double() if st["gate"] is not None else None
    r = st["residual"].double() + _branch64(st, y, st["w_post"], gate)
    n = _norm64(r, st["w_pre"])
    return {"out": y, "r": r, "n": n} if op == "combine_norm" and c["keep"] else {"r": r, "n": n}
