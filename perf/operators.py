"""The operators around the W4A4 linears of a transformer block, as cases to measure:

  linear_w4a16   y = x W^T for a few rows of 16-bit activations, W in 4 bits with one scale (and one offset) per group
  qk_norm_rope   RMS norm of every query and key head and the rotary rotation over several position axes, in one pass
  attention      softmax attention over packed sequences, full or causal, grouped heads, long prompts and single tokens

`run` computes each in its plain form (elementary torch operations in 32 bits) or, where `own` is true, by the
package's own entry points.  `exact` gives the same from the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the smallest matrix-vector product of the square layer: launch latency counts
        {"name": "w4a16 1x3072->3072", "op": "linear_w4a16", "M": 1, "K": 3072, "N": 3072, "group": 128,
         "dtype": "bf16", "offset": False, "bias": False},
        # the modulation projection of a 5120-wide block: one conditioning row to shift, scale and gate of both halves
        {"name": "w4a16 1x5120->30720", "op": "linear_w4a16", "M": 1, "K": 5120, "N": 30720, "group": 64,
         "dtype": "bf16", "offset": False, "bias": True},
        # a decode-like batch through the MLP down projection, weights quantised with offsets
        {"name": "w4a16 8x12288->3072", "op": "linear_w4a16", "M": 8, "K": 12288, "N": 3072, "group": 128,
         "dtype": "fp16", "offset": True, "bias": False},
        # a larger batch through a 5120-wide up projection, small groups
        {"name": "w4a16 16x5120->13824", "op": "linear_w4a16", "M": 16, "K": 5120, "N": 13824, "group": 32,
         "dtype": "bf16", "offset": False, "bias": True},
        # one decoded token at a far position: latency
        {"name": "rope 1 token 32/8 heads", "op": "qk_norm_rope", "grid": "1", "start": 100003, "Hq": 32, "Hk": 8,
         "D": 128, "axes": "128", "theta": 1000000.0, "interleaved": False, "dtype": "bf16", "fused": False},
        # a ragged text prompt with 64-wide heads, part of each head rotated
        {"name": "rope 1001 tokens 32/8 halves", "op": "qk_norm_rope", "grid": "1001", "start": 0, "Hq": 32, "Hk": 8,
         "D": 64, "axes": "32", "theta": 10000.0, "interleaved": False, "dtype": "fp16", "fused": True},
        # 1024^2 image latents of the square layer: 64 x 72 positions, 24 heads, q and k out of one fused buffer
        {"name": "rope image 4608x24", "op": "qk_norm_rope", "grid": "1,64,72", "start": 0, "Hq": 24, "Hk": 24,
         "D": 128, "axes": "16,56,56", "theta": 10000.0, "interleaved": True, "dtype": "bf16", "fused": True},
        # the video latents of the block stack: 21 x 30 x 52 positions, 40 heads
        {"name": "rope video 32760x40", "op": "qk_norm_rope", "grid": "21,30,52", "start": 0, "Hq": 40, "Hk": 40,
         "D": 128, "axes": "44,42,42", "theta": 10000.0, "interleaved": True, "dtype": "bf16", "fused": False},
        # single tokens of eight sequences over caches of different lengths
        {"name": "attention 8 tokens over caches", "op": "attention", "q": "1,1,1,1,1,1,1,1",
         "k": "16384,9001,4096,12345,777,16000,1,8192", "Hq": 32, "Hk": 8, "D": 128, "causal": True, "dtype": "bf16"},
        # packed prompts of different lengths, grouped heads, causal
        {"name": "attention packed prompts", "op": "attention", "q": "4096,1,77,2531,1000,333,3001,129",
         "k": "4096,1,77,2531,1000,333,3001,129", "Hq": 40, "Hk": 8, "D": 128, "causal": True, "dtype": "fp16"},
        # the image latents: every token sees every other
        {"name": "attention image 4608x24", "op": "attention", "q": "4608", "k": "4608", "Hq": 24, "Hk": 24, "D": 128,
         "causal": False, "dtype": "bf16"},
        # the video latents, the ten of forty heads that one of four ranks holds
        {"name": "attention video 32760x10", "op": "attention", "q": "32760", "k": "32760", "Hq": 10, "Hk": 10,
         "D": 128, "causal": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_w4a16", "qk_norm_rope", "attention"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "linear_w4a16":
        group = rng.choice([32, 64, 128])
        K = max(1, _log(rng, 256, 13824) // group) * group
        N = _log(rng, 64, 30720)
        return {"op": op, "M": _log(rng, 1, 16), "K": K, "N": min(N, 5120 * 30720 // K), "group": group, "dtype": dtype,
                "offset": rng.random() < 0.5, "bias": rng.random() < 0.5}
    Hk = rng.choice([1, 2, 4, 5, 8, 10, 12])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4, 5, 8])
    if op == "qk_norm_rope":
        D = rng.choice([64, 96, 128])
        count = rng.choice([1, 2, 3])
        if count == 1:
            grid, axes = str(_log(rng, 1, 32760)), str(rng.choice([D, D // 2]))
        elif count == 2:
            grid, axes = "%d,%d" % (_log(rng, 1, 180), _log(rng, 1, 180)), "%d,%d" % (D // 2, D // 2)
        else:
            grid = "%d,%d,%d" % (_log(rng, 1, 21), _log(rng, 1, 39), _log(rng, 1, 39))
            axes = "%d,%d,%d" % (D - 4 * (D // 6), 2 * (D // 6), 2 * (D // 6))
        return {"op": op, "grid": grid, "start": rng.choice([0, rng.randrange(200000)]), "Hq": Hq, "Hk": Hk, "D": D,
                "axes": axes, "theta": rng.choice([10000.0, 1000000.0]), "interleaved": rng.random() < 0.5,
                "dtype": dtype, "fused": rng.random() < 0.5}
    kind = rng.choice(["full", "causal", "tokens"])
    B = _log(rng, 1, 8)
    most = int(math.sqrt(10 * 32760.0 ** 2 / (B * Hq)))
    ks = [_log(rng, 1, min(most, 16384)) for _ in range(B)]
    if kind == "tokens":
        qs = [min(n, _log(rng, 1, 4)) for n in ks]
    else:
        qs = list(ks)
    return {"op": op, "q": ",".join(map(str, qs)), "k": ",".join(map(str, ks)), "Hq": Hq, "Hk": Hk,
            "D": rng.choice([64, 128]), "causal": kind != "full", "dtype": dtype}


def _ints(text):
    return [int(t) for t in text.split(",")]


def _frequencies(case):
    """freq [R/2] in 64 bits and the axis [R/2] of every rotated pair: theta^(-2 i / d) along each axis of d dims."""
    dims = _ints(case["axes"])
    freq = [case["theta"] ** (-2.0 * i / d) for d in dims for i in range(d // 2)]
    axis = [a for a, d in enumerate(dims) for _ in range(d // 2)]
    return (torch.tensor(freq, dtype=torch.float64, device="cuda"),
            torch.tensor(axis, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    s = {"case": case}
    if case["op"] == "linear_w4a16":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        w = torch.randn(N, K // G, G, generator=gen, device="cuda", dtype=torch.float32).mul_(0.02)
        if case["offset"]:
            lo, hi = w.amin(2, True), w.amax(2, True)
            scale = ((hi - lo) / 15).to(dtype)
            offset = (lo + 8 * scale.float()).to(dtype)
            code = ((w - offset.float()) / scale.float()).round_().clamp_(-8, 7)
            s["offset"] = offset.view(N, K // G)
        else:
            scale = (w.abs().amax(2, True) / 7).to(dtype)
            code = (w / scale.float()).round_().clamp_(-7, 7)
            s["offset"] = None
        code = code.view(N, K).to(torch.int32) & 15
        s["Wq"] = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8).view(torch.int8)
        s["scale"] = scale.view(N, K // G)
        s["x"] = normal(M, K)
        s["bias"] = normal(N) if case["bias"] else None
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "qk_norm_rope":
        grid = _ints(case["grid"])
        T = math.prod(grid)
        if case["fused"]:
            qkv = normal(T, (Hq + 2 * Hk) * D)
            s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
            s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        else:
            s["q"], s["k"] = normal(T, Hq, D), normal(T, Hk, D)
        s["q_weight"], s["k_weight"] = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        axes = [torch.arange(n, device="cuda", dtype=torch.int32) for n in grid]
        s["positions"] = torch.cartesian_prod(*axes).view(T, len(grid)) + case["start"]
        s["freq"], s["axis"] = _frequencies(case)
        return s
    qs, ks = _ints(case["q"]), _ints(case["k"])
    s["q"], s["k"], s["v"] = normal(sum(qs), Hq, D), normal(sum(ks), Hk, D), normal(sum(ks), Hk, D)
    for name, n in (("cu_q", qs), ("cu_k", ks)):
        s[name] = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")
    s["most_q"], s["most_k"] = max(qs), max(ks)
    s["ragged"] = min(ks) < max(ks)
    return s


def _plain_linear(s):
    N = s["Wq"].shape[0]
    b = s["Wq"].view(torch.uint8)
    code = torch.stack((b & 15, b >> 4), 2).view(N, -1).float()
    code = torch.where(code > 7, code - 16, code)
    w = code.view(N, s["scale"].shape[1], -1) * s["scale"].float()[:, :, None]
    if s["offset"] is not None:
        w = w + s["offset"].float()[:, :, None]
    y = s["x"].float() @ w.view(N, -1).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def _plain_rotate(h, weight, cos, sin, interleaved, eps):
    u = h.float()
    u = u * torch.rsqrt(u.square().mean(2, True) + eps) * weight.float()
    R = 2 * cos.shape[1]
    c, t = cos[:, None], sin[:, None]
    if interleaved:
        a, b = u[:, :, 0:R:2], u[:, :, 1:R:2]
        r = torch.stack((a * c - b * t, a * t + b * c), 3).flatten(2)
    else:
        a, b = u[:, :, :R // 2], u[:, :, R // 2:R]
        r = torch.cat((a * c - b * t, a * t + b * c), 2)
    return torch.cat((r, u[:, :, R:]), 2).to(h.dtype)


def _plain_qk_norm_rope(s, eps):
    angle = s["positions"][:, s["axis"].long()].double() * s["freq"]   # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    inter = s["case"]["interleaved"]
    return (_plain_rotate(s["q"], s["q_weight"], cos, sin, inter, eps),
            _plain_rotate(s["k"], s["k_weight"], cos, sin, inter, eps))


def _plain_attention(s):
    """One padded batch: rows and keys past a sequence's end are masked."""
    q, k, v, cq, ck = s["q"], s["k"], s["v"], s["cu_q"].long(), s["cu_k"].long()
    Lq, Lk, B = s["most_q"], s["most_k"], s["cu_q"].numel() - 1
    Tq, Hq, D = q.shape
    Hk, G = k.shape[1], Hq // k.shape[1]
    i = torch.arange(Lq, device=q.device)
    j = torch.arange(Lk, device=q.device)
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    at_q = (cq[:-1, None] + i).clamp(max=Tq - 1)
    at_k = (ck[:-1, None] + j).clamp(max=k.shape[0] - 1)
    qf = (q[at_q].float() * (1.0 / math.sqrt(D))).view(B, Lq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B * Hk, G * Lq, D)
    kf = k[at_k].float().permute(0, 2, 3, 1).reshape(B * Hk, D, Lk)
    vf = v[at_k].float().permute(0, 2, 1, 3).reshape(B * Hk, Lk, D)
    p = torch.bmm(qf, kf).view(B, Hk, G, Lq, Lk)
    if s["case"]["causal"]:
        seen = j <= i[:, None] + (nk - nq)[:, None, None]
        p.masked_fill_(~(seen & (j < nk[:, None, None])).view(B, 1, 1, Lq, Lk), -math.inf)
    elif s["ragged"]:
        p.masked_fill_((j >= nk[:, None]).view(B, 1, 1, 1, Lk), -math.inf)
    top = p.amax(4, True)
    top = torch.where(top == -math.inf, 0.0, top)
    p.sub_(top).exp_()
    total = p.sum(4, True)
    o = torch.bmm(p.view(B * Hk, G * Lq, Lk), vf).view(B, Hq, Lq, D) / total.view(B, Hq, Lq, 1).clamp(min=1e-30)
    lse = (top + total.log()).view(B, Hq, Lq)
    row = torch.arange(Tq, device=q.device)
    seq = torch.searchsorted(cq[1:], row, right=True)
    return o[seq, :, row - cq[seq]].to(q.dtype), lse[seq, :, row - cq[seq]]


def run(state):
    s, case = state, state["case"]
    if case["op"] == "linear_w4a16":
        if own:
            import w4a4_hadamard_rotated_b200 as w4
            return w4.linear_w4a16(s["x"], s["Wq"], s["scale"], offset=s["offset"], bias=s["bias"])
        return _plain_linear(s)
    if case["op"] == "qk_norm_rope":
        if own:
            import w4a4_hadamard_rotated_b200 as w4
            return w4.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["freq"], s["axis"],
                                   interleaved=case["interleaved"], eps=1e-6)
        return _plain_qk_norm_rope(s, 1e-6)
    if own:
        import w4a4_hadamard_rotated_b200 as w4
        return w4.attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"], return_lse=True)
    return _plain_attention(s)


def work(case):
    if case["op"] == "linear_w4a16":
        M, K, N, G = case["M"], case["K"], case["N"], case["group"]
        b = N * K // 2 + 2 * N * (K // G) * (2 if case["offset"] else 1) + 2 * M * K + 2 * M * N
        return {"bytes": b + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "qk_norm_rope":
        grid = _ints(case["grid"])
        T = math.prod(grid)
        # norm: square, sum and two products per element; rotation: four products and two sums per pair
        return {"bytes": 4 * T * (Hq + Hk) * D + 4 * T * len(grid), "flops": 7 * T * (Hq + Hk) * D}
    qs, ks = _ints(case["q"]), _ints(case["k"])
    pairs = 0
    for n, m in zip(qs, ks):
        if case["causal"]:
            least = max(0, m - n + 1)          # keys the first row sees; the last one sees all m
            rows = min(n, m)
            pairs += rows * (least + m) // 2 if n <= m else m * (m + 1) // 2
        else:
            pairs += n * m
    return {"bytes": 2 * D * (2 * sum(qs) * Hq + 2 * sum(ks) * Hk) + 4 * sum(qs) * Hq, "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear_w4a16":
        bits = s["Wq"].to(torch.int64)
        low = ((bits & 15) ^ 8) - 8
        high = bits >> 4                       # arithmetic: the high nibble with its sign
        N, G = bits.shape[0], case["group"]
        w = torch.empty(N, case["K"], dtype=torch.float64, device=bits.device)
        w[:, 0::2], w[:, 1::2] = low.double(), high.double()
        w *= s["scale"].double().repeat_interleave(G, 1)
        if s["offset"] is not None:
            w += s["offset"].double().repeat_interleave(G, 1)
        y = torch.mm(s["x"].double(), w.T)
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "qk_norm_rope":
        D, dims, start = case["D"], _ints(case["axes"]), case["start"]
        grid = torch.stack(torch.meshgrid(*[torch.arange(n, device="cuda") for n in _ints(case["grid"])], indexing="ij"), -1)
        where = grid.reshape(-1, len(dims)).double() + start
        # every pair as one complex number, turned by e^(i angle)
        theta = torch.tensor(case["theta"], dtype=torch.float64, device="cuda")
        angle = torch.cat([where[:, a, None] * torch.pow(theta, -torch.arange(0, d, 2, device="cuda").double() / d)
                           for a, d in enumerate(dims)], 1)
        turn = torch.complex(torch.cos(angle), torch.sin(angle))
        R = sum(dims)
        first = torch.arange(0, R, 2, device="cuda") if case["interleaved"] else torch.arange(R // 2, device="cuda")
        second = first + (1 if case["interleaved"] else R // 2)
        outs = []
        for name in ("q", "k"):
            h = s[name].double()
            h = h / (torch.linalg.vector_norm(h, dim=2, keepdim=True) ** 2 / D + 1e-6).sqrt() * s[name + "_weight"].double()
            z = torch.complex(h[..., first], h[..., second]) * turn[:, None]
            h[..., first], h[..., second] = z.real, z.imag
            outs.append(h)
        return tuple(outs)
    q, k, v = (s[n].double() for n in "qkv")
    G, scale = case["Hq"] // case["Hk"], case["D"] ** -0.5
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n, m in zip(_ints(case["q"]), _ints(case["k"])):
        for h in range(case["Hq"]):
            kk, vv = k[k0:k0 + m, h // G], v[k0:k0 + m, h // G]
            for r in range(0, n, 8192):
                rows = slice(q0 + r, q0 + min(n, r + 8192))
                t = (q[rows, h] @ kk.T) * scale
                if case["causal"]:
                    i = torch.arange(r, min(n, r + 8192), device="cuda")[:, None] + (m - n)
                    t = t.masked_fill(torch.arange(m, device="cuda")[None] > i, -math.inf)
                z = torch.logsumexp(t, 1)
                lse[rows, h] = z
                out[rows, h] = torch.exp(t - torch.where(z == -math.inf, 0.0, z)[:, None]) @ vv
        q0, k0 = q0 + n, k0 + m
    return out, lse
