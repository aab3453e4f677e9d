"""Cases of the operators of a layer over packed prompts: causal attention with grouped
heads, rotary positions with several axes, a linear layer with bias, activation and residual
in its epilogue, and the gated product of two projections.

Each case runs in two ways from the same state: the plain form (elementary torch operations
in 32 bits) and, where ``own`` is true, the library's calls.
"""
import math
import random

import torch

own = False

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a few short questions at once: latency counts
        dict(name="attn_short", op="attn", batch=3, q_min=30, q_max=260, more_min=0, more_max=0,
             Hq=32, Hkv=8, D=128, causal=True, lens=31),
        # a serving batch of ordinary prompts of unlike lengths
        dict(name="attn_batch", op="attn", batch=24, q_min=90, q_max=2700, more_min=0, more_max=0,
             Hq=32, Hkv=8, D=128, causal=True, lens=32),
        # one long document
        dict(name="attn_long", op="attn", batch=1, q_min=16001, q_max=16001, more_min=0,
             more_max=0, Hq=32, Hkv=8, D=128, causal=True, lens=33),
        # prompts behind prefixes whose rows were read out of a cache, heads of 64
        dict(name="attn_prefix", op="attn", batch=6, q_min=300, q_max=1800, more_min=100,
             more_max=1500, Hq=28, Hkv=4, D=64, causal=True, lens=34),
        # one new token of each of 48 sequences, three axes over one spectrum
        dict(name="rope_step", op="rope", tokens=48, Hq=32, Hkv=8, D=128, dims="32,48,48",
             base=1000000.0, halves=True, shared=True, far=30000, low=0, lens=35),
        # text and image tokens of a mixed-resolution batch, each axis its own spectrum
        dict(name="rope_images", op="rope", tokens=30269, Hq=24, Hkv=24, D=128, dims="16,56,56",
             base=10000.0, halves=False, shared=False, far=128, low=-64, lens=36),
        # patches of images in an encoder, height and width, heads of 80
        dict(name="rope_patches", op="rope", tokens=9801, Hq=16, Hkv=16, D=80, dims="40,40",
             base=10000.0, halves=True, shared=False, far=99, low=0, lens=37),
        # output projection of a step of a few tokens, added to the stream
        dict(name="linear_step", op="linear", M=13, N=4096, K=4096, act="none", bias=False,
             residual=True, lens=38),
        # output projection of packed prompts, added to the stream
        dict(name="linear_out", op="linear", M=4741, N=4096, K=4096, act="none", bias=True,
             residual=True, lens=39),
        # first projection of a feed-forward block over one image's tokens
        dict(name="linear_gelu", op="linear", M=6889, N=8192, K=2048, act="gelu_tanh", bias=True,
             residual=False, lens=40),
        # gated feed-forward of a step of single tokens
        dict(name="gated_step", op="gated", M=24, N=11264, K=4096, act="silu", lens=41),
        # the same of a batch of prompts
        dict(name="gated_prompts", op="gated", M=5003, N=11264, K=4096, act="silu", lens=42),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0.0, 0.0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        op = rng.choice(["attn", "attn", "rope", "linear", "linear", "gated"])
        case = dict(op=op, lens=rng.randrange(1 << 30))
        if op == "attn":
            case["Hkv"], G = rng.choice([(8, 4), (4, 7), (2, 6), (1, 8), (12, 1), (20, 1), (5, 3)])
            case["Hq"] = case["Hkv"] * G
            case["D"] = rng.choice([64, 128, 128])
            case["batch"] = _between(rng, 1, 48)
            case["q_max"] = _between(rng, 1, 12000)
            case["q_min"] = rng.randint(0, case["q_max"])
            case["more_min"], case["more_max"] = 0, 0
            if rng.random() < 0.4:               # keys before the prompt's own, or too few
                case["more_max"] = _between(rng, 1, 4000)
                case["more_min"] = rng.choice([0, 0, -(case["q_max"] // 2)])
            case["causal"] = rng.random() < 0.85
            L = _lengths(case)
            if sum(L["q"]) == 0 or sum(L["k"]) == 0:
                continue
        elif op == "rope":
            case["Hkv"], G = rng.choice([(8, 4), (4, 7), (2, 6), (1, 16), (16, 1), (24, 1)])
            case["Hq"] = case["Hkv"] * G
            case["D"] = rng.choice([64, 72, 80, 96, 128, 128, 256])
            case["tokens"] = _between(rng, 1, 40000)
            width = case["D"] if rng.random() < 0.7 else case["D"] // 16 * 8
            cuts = sorted(rng.sample(range(1, width // 2), rng.randint(1, 4) - 1))
            edges = [0] + cuts + [width // 2]
            case["dims"] = ",".join(str(2 * (b - a)) for a, b in zip(edges, edges[1:]))
            case["base"] = rng.choice([100.0, 10000.0, 500000.0, 5000000.0])
            case["halves"], case["shared"] = rng.random() < 0.5, rng.random() < 0.5
            case["far"] = _between(rng, 2, 2000000)
            case["low"] = rng.choice([0, 0, -case["far"] // 2])
        else:
            case["M"] = _between(rng, 1, 16000)
            case["N"], case["K"] = (8 * _between(rng, 8, 2000) for _ in range(2))
            case["act"] = rng.choice(ACTS)
            if op == "linear":
                case["bias"], case["residual"] = rng.random() < 0.5, rng.random() < 0.5
        w = work(case)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return case


def _lengths(case):
    """Per sequence: q queries and k keys."""
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    k = [max(0, n + rng.randint(case["more_min"], case["more_max"])) for n in q]
    return {"q": q, "k": k}


def _dims(case):
    return [int(d) for d in case["dims"].split(",")]


def work(case):
    if case["op"] == "attn":
        L, pairs = _lengths(case), 0
        for lq, lk in zip(L["q"], L["k"]):
            if case["causal"]:
                seen = min(lq, lk)              # queries that see a key; the last sees all lk
                pairs += seen * lk - seen * (seen - 1) // 2
            else:
                pairs += lq * lk
        rows = 2 * sum(L["q"]) * case["Hq"] + 2 * sum(L["k"]) * case["Hkv"]
        return {"bytes": float(rows * case["D"] * 2),
                "flops": float(4 * case["D"] * case["Hq"] * pairs)}
    if case["op"] == "rope":
        values = case["tokens"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": float(4 * values + 4 * case["tokens"] * len(_dims(case))),
                "flops": float(3 * values)}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gated":
        return {"bytes": 2.0 * (M * K + 2 * N * K + M * N), "flops": 4.0 * M * N * K}
    extra = (N if case["bias"] else 0) + (M * N if case["residual"] else 0)
    return {"bytes": 2.0 * (M * K + N * K + M * N + extra), "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + case["lens"] % 7919)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def bf16(x):
        return x.to(torch.bfloat16)

    s = {"case": case}
    if case["op"] in ("attn", "rope"):
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]

    if case["op"] == "attn":
        L = _lengths(case)
        Tq, Tk = sum(L["q"]), sum(L["k"])
        # channels and tokens of unlike size, as rows after a projection have them
        kv = normal(Tk, 2 * Hkv, D) * torch.exp(0.4 * normal(1, 2 * Hkv, D))
        kv = bf16(kv * torch.exp(0.3 * normal(Tk, 1, 1)))
        if L["q"] == L["k"]:
            # slices of a fused projection's output, as a layer has them
            fused = torch.cat([bf16(normal(Tq, Hq, D)), kv], dim=1)
            s["q"], s["k"], s["v"] = fused.split([Hq, Hkv, Hkv], dim=1)
        else:
            s["q"] = bf16(normal(Tq, Hq, D))
            s["k"], s["v"] = kv[:, :Hkv].contiguous(), kv[:, Hkv:].contiguous()
        for n in "qk":
            s["cu_" + n] = torch.tensor([sum(L[n][:b]) for b in range(len(L[n]) + 1)],
                                        dtype=torch.int32, device=dev)
            s["max_" + n] = max(L[n])
        s["lengths"] = L
        s["out"] = torch.zeros(Tq, Hq, D, dtype=torch.bfloat16, device=dev)
    elif case["op"] == "rope":
        T, dims = case["tokens"], _dims(case)
        fused = bf16(normal(T, Hq + 2 * Hkv, D))
        s["q"], s["k"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
        s["dims"] = dims
        s["positions"] = torch.randint(case["low"], case["far"], (len(dims), T), generator=g,
                                       device=dev, dtype=torch.int32)
        s["q_out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = bf16(normal(M, K) * torch.exp(0.3 * normal(M, 1)))
        s["out"] = torch.zeros(M, N, dtype=torch.bfloat16, device=dev)
        if case["op"] == "gated":
            # both projections' weights in one tensor, as they are stored
            s["w"] = bf16(normal(2 * N, K) / math.sqrt(K))
            s["w_gate"], s["w_up"] = s["w"][:N], s["w"][N:]
        else:
            s["w"] = bf16(normal(N, K) / math.sqrt(K))
            s["bias"] = bf16(0.2 * normal(N)) if case["bias"] else None
            s["residual"] = bf16(2.0 * normal(M, N)) if case["residual"] else None
    return s


# ------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "attn":
        return _plain_attention(state)
    if op == "rope":
        return _plain_rope(state)
    return _plain_linear(state) if op == "linear" else _plain_gated(state)


def _own(s, op):
    import packed_varlen_gb300 as pv
    c = s["case"]
    if op == "attn":
        return pv.prompt_attn_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"],
                                  s["max_k"], causal=c["causal"], out=s["out"])
    if op == "rope":
        return pv.rope_axes(s["q"], s["k"], s["positions"], s["dims"], base=c["base"],
                            halves=c["halves"], shared=c["shared"], q_out=s["q_out"],
                            k_out=s["k_out"])
    if op == "linear":
        return pv.linear_act_bf16(s["x"], s["w"], s["bias"], act=c["act"],
                                  residual=s["residual"], out=s["out"])
    return pv.linear_gated_bf16(s["x"], s["w_gate"], s["w_up"], act=c["act"], out=s["out"])


def _plain_attention(s):
    c, L = s["case"], s["lengths"]
    Hkv, D = c["Hkv"], c["D"]
    G, scale = c["Hq"] // Hkv, 1.0 / math.sqrt(D)
    q0 = k0 = 0
    for lq, lk in zip(L["q"], L["k"]):
        k = s["k"][k0:k0 + lk].float().transpose(0, 1)               # [Hkv, lk, D]
        v = s["v"][k0:k0 + lk].float().transpose(0, 1)
        # rows at a time, so that their scores take about a gigabyte
        step = max(1, (1 << 28) // max(1, c["Hq"] * lk))
        for r in range(0, lq, step):
            n = min(step, lq - r)
            rows = slice(q0 + r, q0 + r + n)
            x = s["q"][rows].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
            score = (torch.matmul(x, k.transpose(1, 2)) * scale).view(Hkv, G, n, lk)
            if lk > 0:
                if c["causal"]:
                    i = torch.arange(r, r + n, device=k.device)[:, None]
                    score.masked_fill_(torch.arange(lk, device=k.device) > lk - lq + i, -math.inf)
                score -= score.amax(-1, keepdim=True).clamp(min=-3.0e38)
                score.exp_()
            den = score.sum(-1, keepdim=True)
            y = torch.matmul(score.view(Hkv, G * n, lk), v).view(Hkv, G, n, D)
            y = torch.where(den > 0, y / den, 0.0).permute(2, 0, 1, 3).reshape(n, Hkv * G, D)
            s["out"][rows] = y.to(torch.bfloat16)
        q0, k0 = q0 + lq, k0 + lk
    return s["out"]


def _spectrum(c, dims, device):
    """(theta, axis) of every pair, in 64 bits."""
    width, theta, axis, done = sum(dims), [], [], 0
    for a, d in enumerate(dims):
        for i in range(d // 2):
            at, of = (done + i, width) if c["shared"] else (i, d)
            theta.append(c["base"] ** (-2.0 * at / of))
            axis.append(a)
        done += d // 2
    return (torch.tensor(theta, dtype=torch.float64, device=device),
            torch.tensor(axis, device=device))


def _plain_rope(s):
    c, width = s["case"], sum(s["dims"])
    theta, axis = _spectrum(c, s["dims"], s["q"].device)
    angle = s["positions"][axis].T * theta                          # [T, pairs], 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        x = x.float()
        if c["halves"]:
            a, b = x[..., :width // 2], x[..., width // 2:width]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        else:
            a, b = x[..., :width:2], x[..., 1:width:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        out.copy_(torch.cat([y, x[..., width:]], dim=-1))
    return s["q_out"], s["k_out"]


def _act(v, name):
    if name == "relu":
        return v.clamp(min=0.0)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s):
    y = torch.matmul(s["x"].float(), s["w"].float().T)
    if s["bias"] is not None:
        y += s["bias"].float()
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return s["out"].copy_(y)


def _plain_gated(s):
    x = s["x"].float()
    gate = torch.matmul(x, s["w_gate"].float().T)
    up = torch.matmul(x, s["w_up"].float().T)
    return s["out"].copy_(_act(gate, s["case"]["act"]) * up)


# ------------------------------------------------------------------- exact

def _exact_act(v, name):
    """In 64 bits, by other formulas than the plain form's where there is one."""
    if name == "relu":
        return torch.maximum(v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def _exact_product(x, w):
    """x w^T in 64 bits, some columns at a time."""
    x = x.to(torch.float64)
    return torch.cat([x @ part.to(torch.float64).T for part in w.split(2048)], dim=1)


def exact(case, seed):
    w = work(case)
    if w["flops"] > 6.0e12:               # 64-bit products run at about a TFLOP/s
        return None
    s = prepare(case, seed)
    if case["op"] == "linear":
        y = _exact_product(s["x"], s["w"])
        if s["bias"] is not None:
            y = y + s["bias"].to(torch.float64)
        y = _exact_act(y, case["act"])
        return y if s["residual"] is None else y + s["residual"].to(torch.float64)
    if case["op"] == "gated":
        return _exact_act(_exact_product(s["x"], s["w_gate"]), case["act"]) * \
            _exact_product(s["x"], s["w_up"])
    if case["op"] == "rope":
        outs, dims = [], s["dims"]
        first, width = 0, sum(dims)
        turned = {n: s[n].to(torch.float64).clone() for n in "qk"}
        for a, d in enumerate(dims):
            for i in range(d // 2):
                power = (first + i) / (width / 2) if case["shared"] else i / (d / 2)
                z = s["positions"][a].to(torch.float64) * math.exp(-math.log(case["base"]) * power)
                e, o = (first + i, first + i + width // 2) if case["halves"] else \
                    (2 * (first + i), 2 * (first + i) + 1)
                for n in "qk":
                    x = s[n].to(torch.float64)
                    turned[n][:, :, e] = torch.cos(z)[:, None] * x[:, :, e] - \
                        torch.sin(z)[:, None] * x[:, :, o]
                    turned[n][:, :, o] = torch.sin(z)[:, None] * x[:, :, e] + \
                        torch.cos(z)[:, None] * x[:, :, o]
            first += d // 2
        return turned["q"], turned["k"]
    G, scale = case["Hq"] // case["Hkv"], case["D"] ** -0.5
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["batch"]):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for h in range(case["Hq"]):
            k = s["k"][cu_k[b]:cu_k[b + 1], h // G].to(torch.float64)
            v = s["v"][cu_k[b]:cu_k[b + 1], h // G].to(torch.float64)
            for r in range(0, lq, 4096):
                at = slice(cu_q[b] + r, cu_q[b] + min(r + 4096, lq))
                z = (s["q"][at, h].to(torch.float64) @ k.T) * scale
                if case["causal"]:
                    last = torch.arange(r, r + z.shape[0], device=z.device)[:, None] + lk - lq
                    z = z.masked_fill(torch.arange(lk, device=z.device) > last, -math.inf)
                weight = torch.nan_to_num(torch.softmax(z, dim=-1))   # rows that see no key
                out[at, h] = weight @ v
    return out
