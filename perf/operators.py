"""Timed cases of the decoder-block operators around the W4A16 linear path.

Three operators, each with its plain form (elementary torch operations in fp32) and the calls a
program makes of the library:

* ``int8``: a linear layer in 8-bit integers, fp16 in and out. The activations are scaled by a
  stored 1/s, quantized per token (127 steps of the row's largest magnitude), multiplied with
  int8 weights quantized per output channel, and scaled back.
* ``norm``: the residual update after a block (post-norm, gate, residual scale) and the RMS norm
  before the next one, whose output is divided by the next linear layer's stored s.
* ``moe``: a whole mixture-of-experts layer for a few tokens: router, softmax, top-k, the chosen
  experts' gate/up and down layers in packed 4-bit weights (groups of 128), the weighted sum.

Layer shapes are those of the Llama-2 7B/70B and Llama-3 8B linear layers, or generic.
"""
import math

import torch

own = False

GROUP = 128
PACKED_BYTES = (2048 + 64 + 16) / 4096.0    # packed bytes per weight: codes, scales, zero points


def listed():
    return [
        # one token through an attention output projection: the latency of the smallest call
        {"name": "int8 token 4096x4096", "op": "int8", "M": 1, "N": 4096, "K": 4096, "scaled": True},
        # a batch of sequences decoding together through the fused q/k/v layer
        {"name": "int8 batch 32 qkv", "op": "int8", "M": 32, "N": 12288, "K": 4096, "scaled": True},
        # a short ragged prompt, sizes that no tile divides
        {"name": "int8 ragged prompt", "op": "int8", "M": 333, "N": 5001, "K": 4112, "scaled": False},
        # a long prompt through the fused gate/up layer: compute-bound
        {"name": "int8 prompt 4096 gate/up", "op": "int8", "M": 4096, "N": 28672, "K": 4096, "scaled": True},
        # one token between two blocks: residual add and pre-norm
        {"name": "norm token", "op": "norm", "M": 1, "K": 4096, "post": False, "gate": "none", "scaled": True},
        # a decoding batch of a model with norms on both sides of a block and a channel gate
        {"name": "norm batch sandwich", "op": "norm", "M": 32, "K": 8192, "post": True, "gate": "channel",
         "scaled": True},
        # ragged prompt, gated by token
        {"name": "norm prompt gated", "op": "norm", "M": 1023, "K": 11016, "post": True, "gate": "token",
         "scaled": False},
        # a long prompt: bandwidth-bound
        {"name": "norm prompt 8192", "op": "norm", "M": 8192, "K": 8192, "post": False, "gate": "none",
         "scaled": True},
        # one token, few wide experts
        {"name": "moe token wide experts", "op": "moe", "T": 1, "E": 8, "top": 2, "K": 4096, "I": 14336,
         "renorm": True, "hscale": False},
        # a few tokens, many narrow experts
        {"name": "moe 5 tokens 64 experts", "op": "moe", "T": 5, "E": 64, "top": 6, "K": 2048, "I": 1408,
         "renorm": False, "hscale": False},
        # an odd number of groups in both layers, a scaled intermediate
        {"name": "moe 19 tokens odd groups", "op": "moe", "T": 19, "E": 12, "top": 3, "K": 1152, "I": 640,
         "renorm": True, "hscale": True},
        # the largest batch: every expert is read, several tokens each
        {"name": "moe 32 tokens wide", "op": "moe", "T": 32, "E": 8, "top": 2, "K": 4096, "I": 14336,
         "renorm": True, "hscale": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int8", "norm", "moe"])
    if op == "int8":
        while True:
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 28672), "K": 16 * _log(rng, 8, 1792),
                 "scaled": rng.random() < 0.5}
            if c["M"] * c["N"] * c["K"] <= 4096 * 28672 * 4096:
                return c
    if op == "norm":
        while True:
            c = {"op": op, "M": _log(rng, 1, 16384), "K": 8 * _log(rng, 8, 3584), "post": rng.random() < 0.5,
                 "gate": rng.choice(["none", "channel", "token"]), "scaled": rng.random() < 0.5}
            if c["M"] * c["K"] * (8 + 2 * (c["gate"] == "token")) <= 8192 * 8192 * 8:
                return c
    while True:
        E = rng.choice([4, 8, 16, 32, 60, 64, 128])
        c = {"op": op, "T": _log(rng, 1, 32), "E": E, "top": rng.randint(1, min(8, E)),
             "K": GROUP * _log(rng, 4, 64), "I": GROUP * _log(rng, 4, 112), "renorm": rng.random() < 0.5,
             "hscale": rng.random() < 0.3}
        if E * c["K"] * c["I"] <= 8 * 4096 * 14336:
            return c


def work(case):
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + 2 * M * N + 4 * K * case["scaled"], "flops": 2 * M * N * K}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        gate = {"none": 0, "channel": 2 * K, "token": 2 * M * K}[case["gate"]]
        return {"bytes": 8 * M * K + gate + 2 * K * (1 + case["post"]) + 4 * K * case["scaled"], "flops": 12 * M * K}
    T, E, top, K, I = (case[k] for k in ("T", "E", "top", "K", "I"))
    active = E * (1.0 - (1.0 - top / E) ** T)     # distinct experts that T tokens choose, on average
    return {"bytes": active * 3 * K * I * PACKED_BYTES + 2 * E * K + 4 * T * K + 4 * active * I * case["hscale"],
            "flops": 2 * T * top * 3 * K * I + 2 * T * E * K}


# ---------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """Standard normal with one channel in a hundred twenty times larger, fp16."""
    x = _randn(g, M, K)
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, round(0.01 * K))]
    x[:, cols] *= 20.0
    return x.half()


def _pack(W):
    """W [N, K] fp16 -> (qweight, scales, zeros): 4-bit codes in groups of 128 along K with an fp16
    scale and a 4-bit zero point, in the packed layout (16-row tiles, an even number of groups)."""
    N, K = W.shape
    G, nt = K // GROUP, -(-N // 16)
    g2 = -(-G // 2)
    w = W.float().view(N, G, GROUP)
    lo, hi = w.amin(2, keepdim=True), w.amax(2, keepdim=True)
    S = ((hi - lo).clamp_min(1e-5) / 15).half()
    z = torch.round(-lo / S.float()).clamp(0, 15)
    q = (torch.round(w / S.float()) + z).clamp(0, 15).to(torch.int32).view(N, K)
    Q = torch.zeros((nt * 16, g2 * 2 * GROUP), dtype=torch.int32, device=W.device)
    Q[:N, :K] = q
    Sp = torch.zeros((nt * 16, 2 * g2), dtype=torch.float16, device=W.device)
    Sp[:N, :G] = S.view(N, G)
    Zp = torch.zeros((nt * 16, 2 * g2), dtype=torch.int32, device=W.device)
    Zp[:N, :G] = z.view(N, G).to(torch.int32)
    # n = 16 T + 8 h + r, k = 64 kt + 16 t + 4 s + 2 e1 + e0; nibble h + 2 e1 + 4 e0 of word (T, kt, r, t, s)
    Q = Q.view(nt, 2, 8, 4 * g2, 4, 4, 2, 2).permute(0, 3, 2, 4, 5, 7, 6, 1).reshape(-1, 8)
    words = torch.zeros(Q.shape[0], dtype=torch.int64, device=W.device)
    for j in range(8):
        words |= Q[:, j].to(torch.int64) << (4 * j)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    Sp = Sp.view(nt, 2, 8, 2 * g2).permute(0, 3, 2, 1).reshape(-1)
    Zp = Zp.view(nt, 2, 8, 2 * g2).permute(0, 3, 2, 1).reshape(-1, 2)
    return words, Sp.contiguous(), (Zp[:, 0] | (Zp[:, 1] << 4)).to(torch.uint8)


def _experts(g, E, N, K):
    """E packed N x K layers of N(0, 0.02^2) weights, stacked."""
    q, s, z = zip(*[_pack((_randn(g, N, K) * 0.02).half()) for _ in range(E)])
    return torch.stack(q), torch.stack(s), torch.stack(z)


def _make(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        s = (_randn(g, K).abs() + 0.05).sqrt() if case["scaled"] else None
        x = _activations(g, M, K)
        W = _randn(g, N, K) * 0.02
        W = (W * s if case["scaled"] else W).half().float()
        sw = W.abs().amax(1) / torch.full((), 127.0, device="cuda")
        return {"x": x, "s": s, "wq": torch.round(W / sw[:, None]).to(torch.int8), "sw": sw}
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        gate = None
        if case["gate"] != "none":
            gate = _randn(g, 1 if case["gate"] == "channel" else M, K).half()
        return {"y": _activations(g, M, K), "r": (2 * _randn(g, M, K)).half(), "gate": gate,
                "w": (1 + 0.1 * _randn(g, K)).half(), "post": (1 + 0.1 * _randn(g, K)).half() if case["post"] else None,
                "s": (_randn(g, K).abs() + 0.05).sqrt() if case["scaled"] else None, "alpha": 0.5, "eps": 1e-6}
    T, E, K, I = (case[k] for k in ("T", "E", "K", "I"))
    return {"x": _randn(g, T, K).half(), "router": (_randn(g, E, K) * 0.02).half(),
            "gate_up": _experts(g, E, 2 * I, K), "down": _experts(g, E, K, I),
            "hs": (_randn(g, E, I).abs() + 0.05).sqrt() if case["hscale"] else None}


def prepare(case, seed):
    st = _make(case, seed)
    st["case"] = case
    if own:
        import weight_only_quantization_w4a16_b200 as P
        st["P"] = P
        if case["op"] == "int8":
            st["layer"] = P.AWQInt8Linear(st["wq"], st["sw"], st["s"])
        if case["op"] == "moe":
            st["layer"] = P.AWQMoE(st["router"], st["gate_up"], st["down"], case["I"], case["top"],
                                   renormalize=case["renorm"], h_scale=st["hs"])
    return st


# ---------------------------------------------------------------------------- one pass
def _unpack(packed, N, K):
    """The packed layers as fp32 weights [E, N, K]: (code - zero point) * scale."""
    words, S, Z = packed
    E, nt, g2 = words.shape[0], -(-N // 16), -(-(K // GROUP) // 2)
    nib = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    q = ((words.view(E, nt, 4 * g2, 8, 4, 4, 1) >> nib) & 15).view(E, nt, 4 * g2, 8, 4, 4, 2, 2, 2)
    q = q.permute(0, 1, 8, 3, 2, 4, 5, 7, 6).reshape(E, nt * 16, 2 * g2, GROUP)
    S = S.view(E, nt, 2 * g2, 8, 2).permute(0, 1, 4, 3, 2).reshape(E, nt * 16, 2 * g2, 1).float()
    Z = Z.view(E, nt, 2 * g2, 8, 1).int()
    Z = torch.cat([Z & 15, Z >> 4], 4).permute(0, 1, 4, 3, 2).reshape(E, nt * 16, 2 * g2, 1)
    return ((q - Z) * S).view(E, nt * 16, -1)[:, :N, :K]


def _plain_int8(st):
    x = st["x"].float()
    if st["s"] is not None:
        x = (x / st["s"]).half().float()
    sx = x.abs().amax(1, keepdim=True) / torch.full((), 127.0, device=x.device)
    q = torch.where(sx > 0, torch.round(x / sx), torch.zeros_like(x))
    return ((q * sx) @ (st["wq"].float() * st["sw"][:, None]).t()).half()


def _rms(v, w, eps):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps) * w.float()


def _plain_norm(st):
    t = st["y"].float()
    if st["post"] is not None:
        t = _rms(t, st["post"], st["eps"])
    if st["gate"] is not None:
        t = t * st["gate"].float()
    h = st["r"].float() + st["alpha"] * t
    x = _rms(h, st["w"], st["eps"])
    if st["s"] is not None:
        x = x / st["s"]
    return h.half(), x.half()


def _plain_moe(st):
    c = st["case"]
    x = st["x"].float()
    logits = x @ st["router"].float().t()
    p = torch.softmax(logits, 1)
    ids = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, : c["top"]]   # ties: lowest index
    top = p.gather(1, ids)
    if c["renorm"]:
        top = top / top.sum(1, keepdim=True)
    weight = torch.zeros_like(p).scatter(1, ids, top)                      # [T, E], zero where not chosen
    gu = torch.matmul(x, _unpack(st["gate_up"], 2 * c["I"], c["K"]).transpose(1, 2))   # [E, T, 2 I]
    gate, up = gu[..., : c["I"]], gu[..., c["I"]:]
    h = gate / (1 + torch.exp(-gate)) * up
    if st["hs"] is not None:
        h = h / st["hs"][:, None, :]
    out = torch.matmul(h, _unpack(st["down"], c["K"], c["I"]).transpose(1, 2))         # [E, T, K]
    return (out * weight.t()[:, :, None]).sum(0).half()


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"int8": _plain_int8, "norm": _plain_norm, "moe": _plain_moe}[op](state)
    if op == "norm":
        return state["P"].awq_residual_norm(state["y"], state["r"], state["w"], post_weight=state["post"],
                                            gate=state["gate"], alpha=state["alpha"], eps=state["eps"], s=state["s"])
    return state["layer"](state["x"])


# ---------------------------------------------------------------------------- 64 bits
def _exact_layer(packed, e, N, K):
    """One expert's weights in fp64, code by code from the layout's index rule."""
    words, S, Z = (v[e] for v in packed)
    dev = words.device
    g2 = -(-(K // GROUP) // 2)
    n, k = torch.arange(N, device=dev)[:, None], torch.arange(K, device=dev)[None, :]
    T, h, r = n // 16, (n // 8) % 2, n % 8
    kt, t, s4, e1, e0 = k // 64, (k // 16) % 4, (k // 4) % 4, (k // 2) % 2, k % 2
    q = (words[(T * 4 * g2 + kt) * 128 + (4 * r + t) * 4 + s4] >> (4 * (h + 2 * e1 + 4 * e0))) & 15
    g = torch.arange(K // GROUP, device=dev)[None, :]
    scale = S[(T * 2 * g2 + g) * 16 + 2 * r + h].double()
    zero = (Z[(T * 2 * g2 + g) * 8 + r].int() >> (4 * h)) & 15
    return ((q.view(N, -1, GROUP) - zero[..., None]).double() * scale[..., None]).view(N, K)


def exact(case, seed):
    st = _make(case, seed)
    if case["op"] == "int8":
        x = st["x"].double()
        if st["s"] is not None:     # the definition rounds x / s to fp16 and the step to fp32
            x = (x / st["s"].double()).float().half().double()
        step = (x.abs().max(dim=1).values / 127.0).float().double()
        code = torch.zeros_like(x)
        live = step > 0
        code[live] = (x[live] / step[live, None]).float().double().round()
        acc = code @ st["wq"].double().t()
        return acc * step[:, None] * st["sw"].double()[None, :]
    if case["op"] == "norm":
        y, r = st["y"].double(), st["r"].double()
        K = case["K"]
        if st["post"] is not None:
            y = y / torch.sqrt(y.pow(2).sum(1, keepdim=True) / K + st["eps"]) * st["post"].double()
        if st["gate"] is not None:
            y = y * st["gate"].double()
        h = r + y * st["alpha"]
        x = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / K + st["eps"]) * st["w"].double()
        return h, x if st["s"] is None else x / st["s"].double()
    x = st["x"].double()
    logits = (x @ st["router"].double().t()).cpu()
    out = torch.zeros_like(x)
    chosen = {}
    for t in range(case["T"]):
        row = logits[t].tolist()
        best = sorted(range(case["E"]), key=lambda e: (-row[e], e))[: case["top"]]
        prob = {e: math.exp(row[e] - row[best[0]]) for e in range(case["E"])}
        total = sum(prob[e] for e in (best if case["renorm"] else prob))
        for e in best:
            chosen.setdefault(e, []).append((t, prob[e] / total))
    for e, who in chosen.items():
        rows = torch.tensor([t for t, _ in who], device=x.device)
        share = torch.tensor([p for _, p in who], device=x.device, dtype=torch.float64)
        gu = x[rows] @ _exact_layer(st["gate_up"], e, 2 * case["I"], case["K"]).t()
        g, u = gu[:, : case["I"]], gu[:, case["I"]:]
        h = u * g * torch.sigmoid(g)
        if st["hs"] is not None:
            h = h / st["hs"][e].double()
        out[rows] += share[:, None] * (h @ _exact_layer(st["down"], e, case["K"], case["I"]).t())
    return out
