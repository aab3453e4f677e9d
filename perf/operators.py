"""Cases of the paged K/V cache operators: writing new tokens into the cache
(bf16, or 8-bit rows with a power-of-two scale), reading cached tokens back as
packed rows, and attention of packed new tokens over the cache.

Each case runs in two ways from the same state: the plain form (elementary
torch operations in 32 bits) and, where ``own`` is true, the library's calls.

Cache layout: k and v pages [num_pages, page, Hkv, D]; 8-bit caches keep one
exponent byte per (token, head) row in [num_pages, Hkv, page].  Position p of
sequence b is row p % page of page table[b, p // page].
"""
import math
import random

import torch

own = False

E_MIN, E_MAX, E_BIAS, E_NAN = -100, 7, 127, 255   # exponents of an 8-bit row
SPARE_PAGES = 3                                   # pages that belong to nobody


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token for each of a few short conversations: latency counts
        dict(name="attn_decode_few", op="attn", batch=4, q_min=1, q_max=1, k_min=180, k_max=700,
             chunks=4, Hq=32, Hkv=8, D=128, page=16, cache="bf16", causal=True, lens=11),
        # a serving batch of ordinary contexts, one new token each
        dict(name="attn_decode_batch", op="attn", batch=64, q_min=1, q_max=1, k_min=900,
             k_max=8000, chunks=64, Hq=32, Hkv=8, D=128, page=16, cache="bf16", causal=True,
             lens=12),
        # a large batch over an 8-bit cache, eight query heads to a K/V head
        dict(name="attn_decode_8bit", op="attn", batch=96, q_min=1, q_max=1, k_min=2000,
             k_max=12000, chunks=96, Hq=64, Hkv=8, D=128, page=64, cache="e4m3", causal=True,
             lens=13),
        # one user's long document, one token at a time
        dict(name="attn_decode_long", op="attn", batch=1, q_min=1, q_max=1, k_min=131000,
             k_max=131000, chunks=1, Hq=32, Hkv=8, D=128, page=32, cache="bf16", causal=True,
             lens=14),
        # a chunk of a long prompt over what came before it
        dict(name="attn_chunk", op="attn", batch=1, q_min=2048, q_max=2048, k_min=14000,
             k_max=14000, chunks=1, Hq=32, Hkv=8, D=128, page=64, cache="bf16", causal=True,
             lens=15),
        # two odd chunks over an 8-bit cache, seven query heads to a K/V head
        dict(name="attn_chunk_8bit", op="attn", batch=2, q_min=400, q_max=800, k_min=5000,
             k_max=9000, chunks=2, Hq=28, Hkv=4, D=128, page=32, cache="e4m3", causal=True,
             lens=16),
        # a mixed step: two prompts' chunks beside sequences that answer
        dict(name="attn_mixed", op="attn", batch=24, q_min=200, q_max=500, k_min=300, k_max=3500,
             chunks=2, Hq=32, Hkv=8, D=128, page=16, cache="bf16", causal=True, lens=17),
        # a decoder's tokens over cached encoder states of another length, no causal order
        dict(name="attn_cross", op="attn", batch=16, q_min=1, q_max=60, k_min=700, k_max=1500,
             chunks=16, Hq=20, Hkv=20, D=64, page=64, cache="bf16", causal=False, lens=18),
        # one new token of each sequence of a batch into an 8-bit cache
        dict(name="write_step_8bit", op="write", batch=96, q_min=1, q_max=1, k_min=2000,
             k_max=6000, Hq=64, Hkv=8, D=128, page=64, cache="e4m3", lens=19),
        # whole prompts into an 8-bit cache, from a fused projection's output
        dict(name="write_prompts_8bit", op="write", batch=12, q_min=500, q_max=5000, k_min=0,
             k_max=900, Hq=32, Hkv=8, D=128, page=16, cache="e4m3", lens=20),
        # a shared prefix out of a bf16 cache, to be attended to with its own heads
        dict(name="read_prefix", op="read", batch=3, q_min=300, q_max=1200, k_min=0, k_max=0,
             Hq=32, Hkv=8, D=128, page=16, cache="bf16", lens=21),
        # a batch's contexts out of an 8-bit cache, to be moved to another layout
        dict(name="read_contexts_8bit", op="read", batch=24, q_min=800, q_max=9000, k_min=0,
             k_max=300, Hq=64, Hkv=8, D=128, page=64, cache="e4m3", lens=22),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["attn", "attn", "attn", "write", "read"])
        Hkv, G = rng.choice([(8, 4), (8, 8), (4, 7), (2, 6), (1, 16), (12, 1), (20, 1), (5, 3)])
        D = rng.choice([64, 128, 128])
        case = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128, 256]),
                    cache=rng.choice(["bf16", "e4m3"]), lens=rng.randrange(1 << 30))
        if op == "attn":
            kind = rng.choice(["decode", "decode", "few", "chunk", "mixed"])
            case["causal"] = rng.random() < 0.8
            case["k_max"] = _between(rng, 30, 40000)
            case["k_min"] = rng.randint(0, case["k_max"])
            if kind in ("decode", "few"):
                case["batch"] = _between(rng, 1, 128)
                case["q_min"], case["q_max"] = 1, 1 if kind == "decode" else rng.randint(2, 12)
                case["chunks"] = case["batch"]
            else:
                case["batch"] = _between(rng, 1, 4) if kind == "chunk" else _between(rng, 4, 40)
                case["q_max"] = _between(rng, 20, 2500)
                case["q_min"] = rng.randint(1, case["q_max"])
                case["chunks"] = case["batch"] if kind == "chunk" else rng.randint(1, 3)
            L = _lengths(case)
            scores = case["batch"] * case["Hq"] * max(L["q"]) * max(L["k"]) * 4
            rows = case["batch"] * max(L["k"]) * Hkv * D * 4
            if scores > 6 << 30 or rows > 5 << 30:
                continue
        else:
            case["batch"] = _between(rng, 1, 128)
            case["q_max"] = _between(rng, 1, 9000)
            case["q_min"] = rng.randint(1, case["q_max"])
            case["k_min"], case["k_max"] = 0, _between(rng, 1, 2000)
            if sum(_lengths(case)["q"]) * Hkv > 8 * 110000:
                continue
        w = work(case)
        if w["bytes"] <= 1.2e9 and w["flops"] <= 4.0e11:
            return case


def _lengths(case):
    """Per sequence: q new (or read) tokens, off positions before them, k keys attended to."""
    rng = random.Random(case["lens"])
    q, off, k = [], [], []
    for b in range(case["batch"]):
        lq = 1
        if case["op"] != "attn" or b < case["chunks"]:
            lq = rng.randint(case["q_min"], case["q_max"])
        before = rng.randint(case["k_min"], case["k_max"])
        q.append(lq)
        off.append(before)
        # a causal step's own tokens are in the cache already; cross attention has keys alone
        k.append(before + lq if case.get("causal", True) else max(1, before))
    return {"q": q, "off": off, "k": k}


def work(case):
    L = _lengths(case)
    row = case["D"] * 2 if case["cache"] == "bf16" else case["D"] + 1
    if case["op"] != "attn":
        rows = 2 * sum(L["q"]) * case["Hkv"]
        return {"bytes": float(rows * (row + case["D"] * 2)), "flops": 0.0}
    pairs = 0
    for lq, lk in zip(L["q"], L["k"]):
        pairs += lq * lk - (lq * (lq - 1) // 2 if case["causal"] else 0)
    nbytes = 2 * sum(L["k"]) * case["Hkv"] * row + 2 * sum(L["q"]) * case["Hq"] * case["D"] * 2
    return {"bytes": float(nbytes), "flops": float(4 * case["D"] * case["Hq"] * pairs)}


# ------------------------------------------------------------------- inputs

def _pages_of(x, case):
    """Rows [P, page, Hkv, D] fp32 -> what a cache holds of them: (pages, exponent bytes)."""
    if case["cache"] == "bf16":
        return x.to(torch.bfloat16), None
    payload, byte = _quantise(x)
    return payload, byte.transpose(1, 2).contiguous()


def prepare(case, seed):
    L = _lengths(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + case["lens"] % 7919)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    held = L["k"] if case["op"] == "attn" else [a + b for a, b in zip(L["q"], L["off"])]
    counts = [-(-n // page) for n in held]
    width = max(counts)
    num_pages = sum(counts) + SPARE_PAGES
    # pages are handed out as they come free, so a sequence's pages lie anywhere
    perm = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    start = torch.tensor([sum(counts[:b]) for b in range(len(counts))], device=dev)
    col = torch.arange(width, device=dev)
    table = perm[(start[:, None] + col).clamp(max=num_pages - 1)]
    table = torch.where(col < torch.tensor(counts, device=dev)[:, None], table, -1).contiguous()

    # channels of unlike size, as keys after a projection have them, and tokens of unlike size
    def rows(n):
        x = torch.randn(n, Hkv, D, generator=g, device=dev)
        x *= torch.exp(0.5 * torch.randn(1, Hkv, D, generator=g, device=dev))
        x *= torch.exp(0.4 * torch.randn(n, 1, 1, generator=g, device=dev))
        return x

    s = {"case": case, "table": table, "total": sum(L["q"]),
         "max_q": max(L["q"]), "max_k": max(held)}
    s["cu"] = torch.tensor([sum(L["q"][:b]) for b in range(len(L["q"]) + 1)], dtype=torch.int32,
                           device=dev)
    s["off"] = torch.tensor(L["off"], dtype=torch.int32, device=dev)
    s["seq_lens"] = torch.tensor(L["k"], dtype=torch.int32, device=dev)
    shape = (num_pages, page, Hkv, D)
    s["k_cache"], s["k_exp"] = _pages_of(rows(num_pages * page).view(shape), case)
    s["v_cache"], s["v_exp"] = _pages_of(rows(num_pages * page).view(shape), case)
    T = s["total"]
    if case["op"] == "attn":
        # q is a slice of a fused projection's output, as a layer has it
        fused = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=dev).to(torch.bfloat16)
        s["q"] = fused[:, :Hq * D].view(T, Hq, D)
        s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
    elif case["op"] == "write":
        fused = torch.cat([torch.zeros(T, Hq * D, device=dev), rows(T).view(T, Hkv * D),
                           rows(T).view(T, Hkv * D)], dim=1).to(torch.bfloat16)
        s["k"] = fused[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["v"] = fused[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    else:
        s["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "attn":
        return _plain_attention(state)
    return _plain_write(state) if op == "write" else _plain_read(state)


def _own(s, op):
    import packed_varlen_gb300 as pv
    if op == "attn":
        return pv.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["cu"], s["seq_lens"],
                                 s["table"], s["max_q"], s["max_k"], k_exp=s["k_exp"],
                                 v_exp=s["v_exp"], causal=s["case"]["causal"], out=s["out"])
    if op == "write":
        pv.kv_cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["table"],
                          pos_offset=s["off"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        return _held(s)
    return pv.kv_cache_read(s["k_cache"], s["v_cache"], s["cu"], s["table"], s["total"],
                            pos_offset=s["off"], k_exp=s["k_exp"], v_exp=s["v_exp"],
                            k_out=s["k_out"], v_out=s["v_out"])


def _held(s):
    if s["k_exp"] is None:
        return [s["k_cache"], s["v_cache"]]
    return [s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"]]


def _power(e):
    """2^e in fp32 from its bits, for whole e in [-126, 127]: a power function may be an ulp off."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """fp32 rows [..., D] -> (e4m3 payload, exponent bytes [...]).  a = max |x| = f 2^n with f in
    [1/2, 1); the scale 2^e is the smallest power of two with a 2^-e <= 448 = 7/8 * 2^9."""
    bad = torch.isnan(x).any(-1)
    x = torch.where(bad[..., None], 0.0, x)
    a = x.abs().amax(-1).clamp(max=3.0e38)
    f, n = torch.frexp(a)
    e = torch.where(f > 0.875, n - 8, n - 9)
    e = torch.where(a == 0, E_MIN, e).clamp(E_MIN, E_MAX)
    y = (x * _power(-e)[..., None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn), torch.where(bad, E_NAN, e + E_BIAS).to(torch.uint8)


def _values(payload, byte):
    """e4m3 rows [..., D] and their exponent bytes [...] -> fp32."""
    scale = torch.where(byte == E_NAN, float("nan"), _power(byte.to(torch.int32) - E_BIAS))
    return payload.float() * scale[..., None]


def _places(s):
    """Page and row in it of every packed token."""
    t = torch.arange(s["total"], device=s["cu"].device)
    b = torch.bucketize(t, s["cu"][1:].long(), right=True)
    p = s["off"].long()[b] + t - s["cu"].long()[b]
    page = s["case"]["page"]
    return s["table"][b, p // page].long(), p % page


def _plain_write(s):
    at, row = _places(s)
    for new, pages, exps in ((s["k"], s["k_cache"], s["k_exp"]),
                             (s["v"], s["v_cache"], s["v_exp"])):
        if exps is None:
            pages[at, row] = new
        else:
            payload, byte = _quantise(new.float())
            pages.view(torch.uint8)[at, row] = payload.view(torch.uint8)
            exps[at, :, row] = byte
    return _held(s)


def _plain_read(s):
    at, row = _places(s)
    for out, pages, exps in ((s["k_out"], s["k_cache"], s["k_exp"]),
                             (s["v_out"], s["v_cache"], s["v_exp"])):
        if exps is None:
            out.copy_(pages[at, row])
        else:
            payload = pages.view(torch.uint8)[at, row].view(torch.float8_e4m3fn)
            out.copy_(_values(payload, exps[at, :, row]))
    return s["k_out"], s["v_out"]


def _gathered(pages, exps, table, n):
    """The first n positions of every sequence: [B, Hkv, n, D] fp32."""
    used = table[:, :-(-n // pages.shape[1])].clamp(min=0).long()
    if exps is None:
        x = pages[used].float()
    else:
        x = _values(pages.view(torch.uint8)[used].view(torch.float8_e4m3fn),
                    exps[used].transpose(2, 3))
    B, P, page, Hkv, D = x.shape
    return x.view(B, P * page, Hkv, D)[:, :n].transpose(1, 2)


def _plain_attention(s):
    c, q, cu = s["case"], s["q"], s["cu"].long()
    Hkv, D, nq, nk = c["Hkv"], c["D"], s["max_q"], s["max_k"]
    G, B, dev = c["Hq"] // c["Hkv"], c["batch"], q.device
    lq, lk = cu[1:] - cu[:-1], s["seq_lens"].long()
    i, j = torch.arange(nq, device=dev), torch.arange(nk, device=dev)
    at = (cu[:-1, None] + i).clamp(max=s["total"] - 1)
    x = q[at].float().view(B, nq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, nq * G, D)
    k = _gathered(s["k_cache"], s["k_exp"], s["table"], nk)
    v = _gathered(s["v_cache"], s["v_exp"], s["table"], nk)
    last = (lk[:, None] - 1).expand(B, nq)            # the last key that each query sees
    if c["causal"]:
        last = torch.minimum(last, (lk - lq)[:, None] + i)
    hidden = (j > last[:, :, None])[:, None, :, None, :]
    score = (torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(D))).view(B, Hkv, nq, G, nk)
    score.masked_fill_(hidden, -math.inf)
    score -= score.amax(-1, keepdim=True).clamp(min=-3.0e38)
    score.exp_()
    den = score.sum(-1, keepdim=True)
    y = torch.matmul(score.view(B, Hkv, nq * G, nk), v).view(B, Hkv, nq, G, D)
    y = torch.where(den > 0, y / den, 0.0).permute(0, 2, 1, 3, 4).reshape(B, nq, Hkv * G, D)
    own_row = i < lq[:, None]
    s["out"][at[own_row]] = y[own_row].to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------- exact

def _exact_rows(pages, exps, ids, n):
    """Rows [n, Hkv, D] of one sequence in 64 bits; ids: its pages."""
    x = pages[ids.long()] if exps is None else \
        pages.view(torch.uint8)[ids.long()].view(torch.float8_e4m3fn)
    x = x.to(torch.float64)
    if exps is not None:
        power = exps[ids.long()].permute(0, 2, 1).to(torch.int64) - E_BIAS
        x = x * _exact_power(power)[..., None]
    return x.reshape(-1, *x.shape[2:])[:n]


def _exact_power(e):
    """2^e in 64 bits from its bits, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_e4m3(x, cap=448.0):
    """64-bit rows -> (nearest e4m3 values, exponent): scaled by the least power of two that
    brings the largest magnitude to 448 or less, then rounded to the grid of each binade."""
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2((a / cap).clamp(min=2.0 ** -200))).to(torch.int64)
    for step in (-1, 1):         # the logarithm's own rounding may be one off at a border
        e = torch.where((a > cap * _exact_power(e)) if step > 0 else
                        (a <= cap * _exact_power(e - 1)), e + step, e)
    e = torch.where(a == 0, E_MIN, e).clamp(E_MIN, E_MAX)
    y = x * _exact_power(-e)[..., None]
    size = y.abs().clamp(min=2.0 ** -6)           # e4m3's grid is even below 2^-6
    binade = torch.round(torch.log2(size)).to(torch.int64)
    binade = torch.where(_exact_power(binade) > size, binade - 1, binade)
    grid = _exact_power(binade - 3)
    return (torch.round(y / grid) * grid).clamp(-cap, cap), e


def exact(case, seed):
    s = prepare(case, seed)
    L = _lengths(case)
    page, table = case["page"], s["table"]
    if case["op"] == "write":
        pages = [s["k_cache"].to(torch.float64), s["v_cache"].to(torch.float64)]
        for x, dst in zip((s["k"], s["v"]), pages):
            y = x.to(torch.float64)
            if case["cache"] == "e4m3":
                y, _ = _exact_e4m3(y)
            t0 = 0
            for b, n in enumerate(L["q"]):
                p = torch.arange(L["off"][b], L["off"][b] + n, device=dst.device)
                dst[table[b, p // page].long(), p % page] = y[t0:t0 + n]
                t0 += n
        return pages + ([None, None] if case["cache"] == "e4m3" else [])
    if case["op"] == "read":
        outs = []
        for pages, exps in ((s["k_cache"], s["k_exp"]), (s["v_cache"], s["v_exp"])):
            rows = []
            for b, n in enumerate(L["q"]):
                held = L["off"][b] + n
                ids = table[b, :-(-held // page)]
                rows.append(_exact_rows(pages, exps, ids, held)[L["off"][b]:])
            outs.append(torch.cat(rows))
        return tuple(outs)
    G, D, scale = case["Hq"] // case["Hkv"], case["D"], 1.0 / math.sqrt(case["D"])
    out = torch.zeros(s["total"], case["Hq"], D, dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (lq, lk) in enumerate(zip(L["q"], L["k"])):
        ids = table[b, :-(-lk // page)]
        k = _exact_rows(s["k_cache"], s["k_exp"], ids, lk)
        v = _exact_rows(s["v_cache"], s["v_exp"], ids, lk)
        q = s["q"][t0:t0 + lq].to(torch.float64)
        for h in range(case["Hkv"]):
            z = torch.einsum("qgd,kd->gqk", q[:, h * G:(h + 1) * G], k[:, h]) * scale
            if case["causal"]:
                i = torch.arange(lq, device="cuda")[:, None]
                z.masked_fill_(torch.arange(lk, device="cuda") > lk - lq + i, -math.inf)
            out[t0:t0 + lq, h * G:(h + 1) * G] = torch.einsum(
                "gqk,kd->qgd", torch.softmax(z, dim=-1), v[:, h])
        t0 += lq
    return out
