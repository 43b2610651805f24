"""The linear layers that finish a decoder block, as calls to be timed and compared.

Five operators: the NVFP4 W4A4 product and the INT4 W4A16 product with bias,
activation and residual in their epilogue, the router of a mixture-of-experts
layer, its INT4 experts for a few tokens, and the whole layer.  `run` computes
them in plain torch, in 32 bits, or (`own`) through the package.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
E2M1_MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # o_proj of an 8192-token prefill, added to the residual stream
        {"name": "prefill_o_residual", "op": "w4a4", "M": 8192, "N": 4096, "K": 4096, "act": "none", "bias": False, "residual": True},
        # down_proj of the same prefill: three times the K
        {"name": "prefill_down_residual", "op": "w4a4", "M": 8192, "N": 4096, "K": 12288, "act": "none", "bias": False, "residual": True},
        # a short ragged prefill chunk through a biased layer, no side a whole tile
        {"name": "prefill_ragged_gelu", "op": "w4a4", "M": 777, "N": 5128, "K": 1088, "act": "gelu_tanh", "bias": True, "residual": False},
        # o_proj of one token being decoded
        {"name": "decode_o_one", "op": "w4a16", "M": 1, "N": 4096, "K": 4096, "act": "none", "bias": False, "residual": True},
        # down_proj of a batch of 16
        {"name": "decode_down_16", "op": "w4a16", "M": 16, "N": 4096, "K": 12288, "act": "none", "bias": False, "residual": True},
        # a wide biased layer with an activation at the largest decode batch, one row short
        {"name": "decode_wide_silu_31", "op": "w4a16", "M": 31, "N": 24576, "K": 4096, "act": "silu", "bias": True, "residual": False},
        # the router of one token: latency
        {"name": "route_one", "op": "route", "T": 1, "E": 128, "H": 4096, "k": 8, "renorm": True},
        # the router of a full decode batch over many experts
        {"name": "route_32_wide", "op": "route", "T": 32, "E": 384, "H": 5120, "k": 8, "renorm": False},
        # experts of a batch that the engine padded: the last rows have no expert
        {"name": "experts_13_padded", "op": "experts", "T": 13, "E": 60, "H": 2048, "I": 1408, "k": 4, "residual": True, "pad": 3},
        # few large experts, every one of them met by several tokens
        {"name": "experts_32_large", "op": "experts", "T": 32, "E": 8, "H": 4096, "I": 12288, "k": 2, "residual": True, "pad": 0},
        # the whole layer for one token: small experts, latency
        {"name": "moe_one", "op": "moe", "T": 1, "E": 128, "H": 2048, "I": 768, "k": 8, "residual": True, "renorm": True},
        # the whole layer for a full decode batch: most experts are read
        {"name": "moe_32", "op": "moe", "T": 32, "E": 128, "H": 4096, "I": 1408, "k": 8, "residual": True, "renorm": True},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(("w4a4", "w4a16", "route", "experts", "moe"))
    if op == "w4a4":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 64, 4096, 8), "K": _log_int(rng, 64, 12288, 64),
                "act": rng.choice(ACTS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.6}
    if op == "w4a16":
        return {"op": op, "M": _log_int(rng, 1, 32), "N": _log_int(rng, 64, 24576, 32), "K": _log_int(rng, 128, 12288, 128),
                "act": rng.choice(ACTS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.6}
    if op == "route":
        E = _log_int(rng, 4, 512)
        return {"op": op, "T": _log_int(rng, 1, 64), "E": E, "H": _log_int(rng, 256, 8192, 64), "k": rng.randint(1, min(8, E)),
                "renorm": rng.random() < 0.5}
    E = _log_int(rng, 4, 128)
    c = {"op": op, "T": _log_int(rng, 1, 32), "E": E, "H": _log_int(rng, 256, 4096, 128), "I": _log_int(rng, 128, 1408, 128),
         "k": rng.randint(1, min(8, E)), "residual": rng.random() < 0.7}
    if op == "experts":
        c["pad"] = rng.randint(0, c["T"] // 2)
    else:
        c["renorm"] = rng.random() < 0.5
    return c


def _active(c):
    """Experts that a batch is expected to meet."""
    t = c["T"] - c.get("pad", 0)
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** t)


def work(case):
    c = case
    if c["op"] in ("w4a4", "w4a16"):
        M, N, K = c["M"], c["N"], c["K"]
        io = 2 * M * N * (2 if c["residual"] else 1) + (2 * N if c["bias"] else 0)
        if c["op"] == "w4a4":
            return {"bytes": (M + N) * K * 9 // 16 + io, "flops": 2 * M * N * K}
        return {"bytes": N * K // 2 + 2 * N * (K // 128) + 2 * M * K + io, "flops": 2 * M * N * K}
    T, E, H, k = c["T"], c["E"], c["H"], c["k"]
    route = {"bytes": 2 * E * H + 2 * T * H + 8 * T * k, "flops": 2 * T * E * H}
    if c["op"] == "route":
        return route
    weights = _active(c) * 3 * H * c["I"] * (0.5 + 2 / 128)
    rows = (T - c.get("pad", 0)) * k
    w = {"bytes": weights + 2 * T * H * (3 if c["residual"] else 2) + 8 * T * k, "flops": 2 * rows * 3 * H * c["I"]}
    if c["op"] == "moe":
        w = {"bytes": w["bytes"] + 2 * E * H, "flops": w["flops"] + route["flops"]}
    return w


# ------------------------------------------------------------------ inputs
def _activations(M, K, gen):
    """N(0, 1) with 0.1 % of the channels 20 times as large."""
    x = torch.randn(M, K, generator=gen, device=DEV)
    x[:, torch.randperm(K, generator=gen, device=DEV)[:max(1, round(0.001 * K))]] *= 20
    return x.to(torch.bfloat16)


def _nvfp4(x):
    """bf16 [R, K] -> packed E2M1 codes, E4M3 block scales [R, K/16] as bytes, tensor scale."""
    R, K = x.shape
    t = (x.abs().amax().float() / 2688).reshape(1)
    b = x.float().view(R, K // 16, 16)
    s = (b.abs().amax(2) / (6 * t)).clamp(max=448).to(torch.float8_e4m3fn)
    q = b / (s.float() * t).clamp(min=1e-30).unsqueeze(2)
    mid = torch.tensor(E2M1_MID, device=DEV)
    code = (torch.bucketize(q.abs(), mid) + 8 * (q < 0)).to(torch.uint8).view(R, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(torch.uint8), t


def _tile_scales(s):
    """[R, K/16] scale bytes in the 128 x 4 atoms that the block-scaled product reads, rows padded with zeros."""
    R, KB = s.shape
    P = (R + 127) // 128 * 128
    p = torch.zeros(P, KB, dtype=torch.uint8, device=DEV)
    p[:R] = s
    return p.view(P // 128, 4, 32, KB // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _int4(R, K, gen):
    """INT4 codes 0 .. 15 (value + 8) of group-quantized N(0, 0.02^2) weights, and their bf16 scales."""
    u = torch.randn(R, K, generator=gen, device=DEV, dtype=torch.float16).mul_(2.6).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    s = (0.02 / 2.6) * (1 + 0.1 * torch.randn(R, K // 128, generator=gen, device=DEV))
    return u, s.to(torch.bfloat16)


def _pack_int4(u, s):
    """Codes and scales in the decode kernels' order: units of 32 rows x 128 columns."""
    R, K = u.shape
    v = u.view(R // 32, 2, 2, 8, K // 128, 4, 4, 2, 2, 2)          # unit row, tt, hi, g, group, c, q, jj, rh, rl
    b = v[:, :, 0] | (v[:, :, 1] << 4)                              # unit row, tt, g, group, c, q, jj, rh, rl
    codes = b.permute(0, 3, 5, 2, 4, 6, 1, 8, 7).reshape(-1).contiguous()
    scales = s.view(R // 32, 2, 2, 8, K // 128).permute(0, 4, 3, 1, 2).reshape(-1).contiguous()
    return codes, scales.view(torch.uint8)


def _stack_int4(E, R, K, gen):
    """E stacked [R, K] INT4 matrices: row-major codes (two per byte), scales, and the packed form of the stack."""
    codes = torch.empty(E, R, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, R, K // 128, dtype=torch.bfloat16, device=DEV)
    pc = torch.empty(E, R * K // 2, dtype=torch.uint8, device=DEV)
    ps = torch.empty(E, R * (K // 128) * 2, dtype=torch.uint8, device=DEV)
    for e in range(E):
        u, s = _int4(R, K, gen)
        codes[e] = u[:, 0::2] | (u[:, 1::2] << 4)
        scales[e] = s
        pc[e], ps[e] = _pack_int4(u, s)
    return {"codes": codes, "scales": scales, "packed": (pc.view(-1), ps.view(-1))}


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def bf16(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)

    st = {"case": c}
    if c["op"] in ("w4a4", "w4a16"):
        M, N, K = c["M"], c["N"], c["K"]
        if c["op"] == "w4a4":
            xc, xs, xt = _nvfp4(_activations(M, K, gen))
            wc, ws, wt = _nvfp4(bf16(N, K, scale=0.02))
            st["x"], st["w"] = (xc, _tile_scales(xs), xt), (wc, _tile_scales(ws), wt)
            st["x_scales"], st["w_scales"] = xs, ws                  # the same scales in row order, for the plain form
        else:
            st["x"] = _activations(M, K, gen)
            st["w"] = _stack_int4(1, N, K, gen)
        st["bias"] = bf16(N) if c["bias"] else None
        st["residual"] = bf16(M, N) if c["residual"] else None
        st["y"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        return st
    T, E, H, k = c["T"], c["E"], c["H"], c["k"]
    st["x"] = _activations(T, H, gen)
    st["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    st["weights"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
    if c["op"] in ("route", "moe"):
        st["router"] = bf16(E, H, scale=0.02)
    if c["op"] in ("experts", "moe"):
        I = c["I"]
        # gate and up rows of an expert in turn, 16 rows of each
        st["gate_up"] = _stack_int4(E, 2 * I, H, gen)
        st["down"] = _stack_int4(E, H, I, gen)
        st["residual"] = bf16(T, H) if c["residual"] else None
        st["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    if c["op"] == "experts":
        score = torch.rand(T, E, generator=gen, device=DEV)
        ids = score.argsort(dim=1)[:, :k].to(torch.int32)
        ids[T - c["pad"]:] = -1                                      # padded rows have no expert
        st["ids"] = ids.contiguous()
        st["weights"] = torch.softmax(torch.randn(T, k, generator=gen, device=DEV), 1)
    return st


# ------------------------------------------------------------------ the plain forms
def _nvfp4_values(codes, scales, t):
    grid = torch.tensor(E2M1, device=DEV)
    both = torch.stack((codes & 15, codes >> 4), dim=2)
    v = grid[both.long()].view(codes.shape[0], -1, 16)
    return (v * (scales.view(torch.float8_e4m3fn).float() * t).unsqueeze(2)).flatten(1)


def _int4_values(codes, scales):
    """[..., R, K/2] codes -> [..., R, K] fp32."""
    both = torch.stack((codes & 15, codes >> 4), dim=-1).float() - 8
    return (both.view(*scales.shape, 128) * scales.float().unsqueeze(-1)).flatten(-2)


def _activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _plain_linear(st):
    c = st["case"]
    if c["op"] == "w4a4":
        x = _nvfp4_values(st["x"][0], st["x_scales"], st["x"][2])
        w = _nvfp4_values(st["w"][0], st["w_scales"], st["w"][2])
    else:
        x = st["x"].float()
        w = _int4_values(st["w"]["codes"][0], st["w"]["scales"][0])
    v = x @ w.t()
    if st["bias"] is not None:
        v = v + st["bias"].float()
    v = _activate(v, c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(torch.bfloat16)


def _plain_route(st):
    """Logits in 64 bits: which expert is chosen is decided next to a border."""
    c = st["case"]
    logits = st["x"].double() @ st["router"].double().t()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :c["k"]], ids[:, :c["k"]]
    e = torch.exp(top - top[:, :1])
    total = e.sum(1, keepdim=True) if c["renorm"] else torch.exp(logits - top[:, :1]).sum(1, keepdim=True)
    return ids.to(torch.int32), (e / total).float()


def _plain_experts(st, ids, weights):
    """By (token, choice) where there are fewer of those than experts, else every expert for every token."""
    c = st["case"]
    T, E, H, I, k = c["T"], c["E"], c["H"], c["I"], c["k"]
    x = st["x"].float()
    valid = (ids >= 0) & (ids < E)
    safe = torch.where(valid, ids, 0).long()
    wt = torch.where(valid, weights, 0.0)
    pairs = T * k < E
    pick = safe.flatten() if pairs else slice(None)
    gu = _int4_values(st["gate_up"]["codes"][pick], st["gate_up"]["scales"][pick])
    xe = x.repeat_interleave(k, 0).unsqueeze(1) if pairs else x.expand(E, T, H)
    a = torch.bmm(xe, gu.transpose(1, 2)).view(gu.shape[0], -1, I // 16, 2, 16)
    del gu
    gate, up = a[:, :, :, 0].flatten(2), a[:, :, :, 1].flatten(2)
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(h, _int4_values(st["down"]["codes"][pick], st["down"]["scales"][pick]).transpose(1, 2))
    if pairs:
        out = (y.view(T, k, H) * wt.unsqueeze(2)).sum(1)
    else:
        dense = torch.zeros(T, E, device=DEV).scatter_add_(1, safe, wt)
        out = (y * dense.t().unsqueeze(2)).sum(0)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return out.to(torch.bfloat16)


def run(state):
    st, c = state, state["case"]
    if own:
        import phase_disaggregated_quantized_b200 as nvq
        if c["op"] == "w4a4":
            return nvq.nvfp4_gemm_w4a4_epilogue(st["x"], st["w"], c["M"], c["N"], c["K"], bias=st["bias"],
                                                activation=c["act"], residual=st["residual"], y=st["y"])
        if c["op"] == "w4a16":
            pc, ps = st["w"]["packed"]
            return nvq.w4a16_gemm_epilogue(st["x"], pc, ps, c["N"], bias=st["bias"], activation=c["act"],
                                           residual=st["residual"], y=st["y"])
        if c["op"] == "route":
            return nvq.moe_route(st["x"], st["router"], c["k"], renormalize=c["renorm"], ids=st["ids"],
                                 weights=st["weights"])
        if c["op"] == "experts":
            return nvq.w4a16_moe_experts(st["x"], st["ids"], st["weights"], st["gate_up"]["packed"],
                                         st["down"]["packed"], c["E"], c["I"], residual=st["residual"], y=st["y"])
        return nvq.w4a16_moe(st["x"], st["router"], st["gate_up"]["packed"], st["down"]["packed"], c["I"], c["k"],
                             renormalize=c["renorm"], residual=st["residual"], ids=st["ids"], weights=st["weights"],
                             y=st["y"])
    if c["op"] in ("w4a4", "w4a16"):
        return _plain_linear(st)
    if c["op"] == "route":
        return _plain_route(st)
    if c["op"] == "experts":
        return _plain_experts(st, st["ids"], st["weights"])
    ids, weights = _plain_route(st)
    return _plain_experts(st, ids, weights), ids, weights


# ------------------------------------------------------------------ 64 bits
def _exact_act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        z = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return v * torch.special.expit(z)
    if act == "silu":
        return v * torch.special.expit(v)
    return v


def _exact_int4(codes, scales):
    R, K = codes.shape[0], codes.shape[1] * 2
    w = torch.empty(R, K, dtype=torch.float64, device=DEV)
    w[:, 0::2] = (codes % 16).double()
    w[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    return (w - 8) * scales.double().repeat_interleave(128, dim=1)


def _exact_nvfp4(codes, scales, t):
    R, K = codes.shape[0], codes.shape[1] * 2
    c = torch.empty(R, K, dtype=torch.int32, device=DEV)
    c[:, 0::2] = (codes % 16).int()
    c[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").int()
    e, m = (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    s = scales.int()
    se, sm = (s // 8) % 16, (s % 8).double()
    sv = torch.where(se == 0, sm * 2.0 ** -9, (1 + sm / 8) * torch.pow(2.0, (se - 7).double()))
    return torch.where(c >= 8, -mag, mag) * sv.repeat_interleave(16, dim=1) * t.double()


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] in ("w4a4", "w4a16"):
        if c["op"] == "w4a4":
            x = _exact_nvfp4(st["x"][0], st["x_scales"], st["x"][2])
            w = _exact_nvfp4(st["w"][0], st["w_scales"], st["w"][2])
        else:
            x, w = st["x"].double(), _exact_int4(st["w"]["codes"][0], st["w"]["scales"][0])
        v = torch.mm(x, w.T)
        v = _exact_act(v if st["bias"] is None else v + st["bias"].double(), c["act"])
        return v if st["residual"] is None else v + st["residual"].double()
    T, E, k = c["T"], c["E"], c["k"]
    ids, weights = st["ids"], st["weights"].double()
    if c["op"] in ("route", "moe"):
        p = torch.mm(st["x"].double(), st["router"].double().T)
        order = torch.argsort(-p, dim=1, stable=True)[:, :k]
        prob = torch.softmax(p, dim=1).gather(1, order)
        weights = prob / prob.sum(1, keepdim=True) if c["renorm"] else prob
        ids = order.int()
        if c["op"] == "route":
            return ids, weights
    y = torch.zeros(T, c["H"], dtype=torch.float64, device=DEV)
    x, I = st["x"].double(), c["I"]
    for e in range(E):
        share = torch.where(ids == e, weights, torch.zeros_like(weights)).sum(1)
        met = share.nonzero().flatten()
        if met.numel() == 0:
            continue
        w = _exact_int4(st["gate_up"]["codes"][e], st["gate_up"]["scales"][e]).view(I // 16, 2, 16, c["H"])
        g = x[met] @ w[:, 0].reshape(I, -1).T
        u = x[met] @ w[:, 1].reshape(I, -1).T
        h = _exact_act(g, "silu") * u * share[met, None]
        y[met] += h @ _exact_int4(st["down"]["codes"][e], st["down"]["scales"][e]).T
    if st["residual"] is not None:
        y = y + st["residual"].double()
    return (y, ids, weights) if c["op"] == "moe" else y
