"""Cases, plain forms and 64-bit definitions of the attention half of a decoder block: projections with
group-quantized weights, the append of rotated keys and values to a paged 8-bit cache, and attention
over that cache.

Layer widths are those of the workload shapes in workloads/configs.py (hidden 1024, 4096, 5120, 7168);
head counts are the usual ones for such widths with 64- or 128-wide heads.
"""
import math

import torch

own = False

E4M3_MAX_MANTISSA = 1.75  # 448 = 1.75 * 2^8
MIN_SCALE_EXP = -100
NOT_USED = 3072           # no drawn size takes this value


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a small projection: a call that is all latency
        {"name": "linear w4 t1 1024x1024", "op": "linear", "T": 1, "K": 1024, "N": 1024, "bits": 4,
         "group": 128, "bias": False, "residual": False, "pad": 0},
        # q/k/v of a 4096-wide layer (32 + 2 x 8 heads) at 8 bits, a decode batch
        {"name": "linear w8 t16 4096x6144", "op": "linear", "T": 16, "K": 4096, "N": 6144, "bits": 8,
         "group": 128, "bias": False, "residual": False, "pad": 0},
        # output projection with residual of a 5120-wide layer, an odd batch between decode and prompt
        {"name": "linear w4 t37 5120x5003", "op": "linear", "T": 37, "K": 5120, "N": 5003, "bits": 4,
         "group": 64, "bias": True, "residual": True, "pad": 40},
        # q/k/v of a 7168-wide layer (56 + 2 x 8 heads) over a prompt batch
        {"name": "linear w4 t4096 7168x9216", "op": "linear", "T": 4096, "K": 7168, "N": 9216, "bits": 4,
         "group": 128, "bias": False, "residual": False, "pad": 0},
        # one new token for each of 16 sequences
        {"name": "append b16 q1", "op": "append", "n_seq": 16, "new": 1, "old": 2000, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "rot": 128, "neighbours": False, "ragged": True},
        # short pieces on short contexts, 64-wide heads, half of each head rotated, small pages
        {"name": "append b7 ragged d64", "op": "append", "n_seq": 7, "new": 61, "old": 50, "Hq": 16, "Hkv": 4,
         "D": 64, "page": 16, "rot": 32, "neighbours": True, "ragged": True},
        # prompts entering the cache
        {"name": "append b3 prompts", "op": "append", "n_seq": 3, "new": 4096, "old": 100, "Hq": 56, "Hkv": 8,
         "D": 128, "page": 64, "rot": 128, "neighbours": False, "ragged": True},
        # the first tokens of an answer: one short sequence
        {"name": "attention b1 q1 l200", "op": "attention", "n_seq": 1, "new": 1, "len": 200, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "window": 0, "ragged": False},
        # a decode batch of mixed lengths
        {"name": "attention b16 q1 l8192", "op": "attention", "n_seq": 16, "new": 1, "len": 8192, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "window": 0, "ragged": True},
        # one sequence with a very long cache
        {"name": "attention b1 q1 l131072", "op": "attention", "n_seq": 1, "new": 1, "len": 131072, "Hq": 64,
         "Hkv": 8, "D": 128, "page": 128, "window": 0, "ragged": False},
        # pieces of prompts and single tokens in one batch, 64-wide heads, a sliding window, an empty sequence
        {"name": "attention b6 mixed window", "op": "attention", "n_seq": 6, "new": 333, "len": 2500, "Hq": 28,
         "Hkv": 4, "D": 64, "page": 16, "window": 700, "ragged": True},
        # a piece of a long prompt
        {"name": "attention b1 q2048 l8192", "op": "attention", "n_seq": 1, "new": 2048, "len": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == NOT_USED else v


def draw(rng):
    op = rng.choice(["linear", "append", "attention"])
    if op == "linear":
        group = rng.choice([64, 128, 128, 256])
        K = group * _log_int(rng, 512 // group, 7168 // group)
        return {"op": "linear", "T": _log_int(rng, 1, 3000), "K": K + group if K == NOT_USED else K,
                "N": _log_int(rng, 200, 9000), "bits": rng.choice([4, 8]), "group": group,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "pad": 8 * rng.randint(0, 5)}
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    heads = {"Hq": Hkv * rng.choice([1, 3, 4, 7, 8, 16] if Hkv < 8 else [1, 2, 4, 5]), "Hkv": Hkv, "D": D,
             "page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        n_seq = _log_int(rng, 1, 40)
        return {"op": "append", "n_seq": n_seq, "new": _log_int(rng, 1, max(2, 8000 // n_seq)),
                "old": rng.choice([0, _log_int(rng, 1, 1500)]), **heads,
                "rot": rng.choice([D, D, D // 2]), "neighbours": rng.random() < 0.3, "ragged": True}
    if rng.random() < 0.5:  # single tokens, or a few
        n_seq = _log_int(rng, 1, 32)
        length = _log_int(rng, 16, 65536 // n_seq)
        return {"op": "attention", "n_seq": n_seq, "new": min(length, rng.choice([1, 1, 1, 2, 5])), "len": length,
                **heads, "window": rng.choice([0, 0, 0, 300]), "ragged": n_seq > 1}
    n_seq = _log_int(rng, 1, 6)
    length = _log_int(rng, 64, 5000 // n_seq)
    return {"op": "attention", "n_seq": n_seq, "new": _log_int(rng, 8, min(length, 1500)), "len": length, **heads,
            "window": rng.choice([0, 0, 200]), "ragged": n_seq > 1}


def _lengths(case):
    """(tokens in the cache before, new tokens) of each sequence, from the case alone."""
    rows = []
    for s in range(case["n_seq"]):
        part = ((s * 7 + 3) % 11 + 1) / 11.0 if case["ragged"] and s else 1.0
        if case["op"] == "append":
            rows.append((int(case["old"] * part), max(1, int(case["new"] * part))))
        else:
            total = max(1, int(case["len"] * part))
            if case["ragged"] and s == 2:          # one sequence has one new token,
                rows.append((total - 1, 1))
            elif case["ragged"] and s == 4:        # and one has no tokens at all in the cache
                rows.append((0, 0))
            else:
                new = min(total, max(1, int(case["new"] * part)))
                rows.append((total - new, new))
    return rows


def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        b = N * K * case["bits"] // 8 + 2 * N * K // case["group"] + 2 * T * (K + N)
        b += 4 * N * case["bias"] + 2 * T * N * case["residual"]
        return {"bytes": b, "flops": 2 * T * N * K}
    rows = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(n for _, n in rows)
    if case["op"] == "append":
        # q in and out, k and v in, codes out, the table's rows, slots and positions, a scale pair a page
        pages = sum(-(-(o + n) // case["page"]) - o // case["page"] for o, n in rows)
        return {"bytes": T * (4 * Hq * D + 6 * Hkv * D + 4 * case["rot"] + 8) + 8 * pages * Hkv,
                "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * T * Hkv * D}
    kv = pairs = 0
    for o, n in rows:
        if n:
            first = max(0, o - case["window"] + 1) if case["window"] else 0
            kv += o + n - first
            if case["window"]:
                pairs += sum(min(o + i + 1, case["window"]) for i in range(n))
            else:
                pairs += n * o + n * (n + 1) // 2
    return {"bytes": kv * Hkv * 2 * D + 8 * (kv // case["page"]) * Hkv + 4 * T * Hq * D,
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = {"device": "cuda", "generator": g}
    bf16 = torch.bfloat16
    s = {"case": dict(case)}
    if case["op"] == "linear":
        T, K, N, G = case["T"], case["K"], case["N"], case["group"]
        if case["bits"] == 4:
            s["codes"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, **dev)
        else:  # int8 codes of normal weights: absmax / 127 is about a third of a standard deviation of 40
            s["codes"] = (torch.randn(N, K, **dev) * 40).round_().clamp_(-127, 127).to(torch.int8)
        s["scales"] = ((torch.rand(N, K // G, **dev) + 0.5) * (0.02 * 3 / (7 if case["bits"] == 4 else 127))).half()
        s["x"] = torch.randn(T, K + case["pad"], **dev).to(bf16)[:, :K]
        s["bias"] = torch.randn(N, **dev) * 0.5 if case["bias"] else None
        s["residual"] = torch.randn(T, N, **dev).to(bf16) if case["residual"] else None
        s["out"] = torch.empty(T, N, dtype=bf16, device="cuda")
        return s

    rows = _lengths(case)
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["page"]
    B, T = len(rows), sum(n for _, n in rows)
    need = [-(-(o + n) // P) for o, n in rows]
    n_pages = sum(need) + 3                               # a few pages that no sequence holds
    order = torch.randperm(n_pages, **dev).to(torch.int32)  # a sequence's pages lie anywhere
    old = torch.tensor([o for o, _ in rows], dtype=torch.int32, device="cuda")
    new = torch.tensor([n for _, n in rows], dtype=torch.int32, device="cuda")
    first_page = torch.tensor([sum(need[:i]) for i in range(B)], dtype=torch.int32, device="cuda")
    most = max(1, max(need))
    col = torch.arange(most, dtype=torch.int32, device="cuda")
    table = order[(first_page[:, None] + col[None]).clamp_max(n_pages - 1).long()].contiguous()
    s["n_pages"] = n_pages
    # codes and scales as an append leaves them
    s["k_codes"] = (torch.randn(n_pages, Hkv, P, D, **dev) * 70).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s["v_codes"] = (torch.randn(n_pages, Hkv, P, D, **dev) * 70).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s["k_scales"] = torch.exp2(torch.randint(-7, -5, (n_pages, Hkv), **dev).float())
    s["v_scales"] = torch.exp2(torch.randint(-8, -5, (n_pages, Hkv), **dev).float())
    s["table"], s["kv_len"], s["n_q"] = table, old + new, new
    start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.cumsum(new, 0)
    s["q_start"], s["T"] = start, T
    s["max_q"], s["max_kv"] = max(n for _, n in rows), max(o + n for o, n in rows)
    # each row's sequence and position, as a scheduler lists them
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new.long(), output_size=T)
    pos = torch.arange(T, device="cuda") - start[seq].long() + old[seq].long()
    s["seq"], s["positions"] = seq, pos.to(torch.int32)
    if case["op"] == "append":
        # q, k and v are column ranges of one projection's output
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, **dev)
        qkv[:, Hq * D:] *= torch.exp(torch.randn(T, 1, **dev) * 0.5)
        qkv = qkv.to(bf16)
        s["q"], s["k"], s["v"] = (qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:])
        s["slots"] = (table[seq, pos // P].long() * P + pos % P).to(torch.int32)
        s["pages"] = torch.unique(s["slots"].long() // P)
        R = case["rot"]
        freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        ang = torch.arange(s["max_kv"], dtype=torch.float64, device="cuda")[:, None] * freq[None]
        s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["q_out"] = torch.empty(T, Hq * D, dtype=bf16, device="cuda")
    else:
        s["q"] = (torch.randn(T, Hq * D, **dev) * 1.5).to(bf16)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty(T, Hq * D, dtype=bf16, device="cuda")
    return s


# ---------------------------------------------------------------------------------------- passes

def run(s):
    op = s["case"]["op"]
    if own:
        return {"linear": _own_linear, "append": _own_append, "attention": _own_attention}[op](s)
    return {"linear": _plain_linear, "append": _plain_append, "attention": _plain_attention}[op](s)


def _own_linear(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    if "lin" not in s:
        s["lin"] = st.QuantLinear(s["codes"], s["scales"], N=c["N"], K=c["K"], bits=c["bits"], group=c["group"],
                                  bias=s["bias"])
        n = s["lin"].workspace_size(c["T"])
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    st.check(st.strata_linear_forward(s["lin"].struct(), s["x"], c["T"], s["out"], s["ws"], s["ws"].numel(),
                                      x_stride=s["x"].stride(0), residual=s["residual"]), "strata_linear_forward")
    return s["out"]


def _own_cache(st, s):
    if "cache" not in s:
        c = s["case"]
        s["cache"] = st.PagedKVCache(s["n_pages"], c["Hkv"], c["D"], c["page"], k_codes=s["k_codes"],
                                     v_codes=s["v_codes"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    return s["cache"].struct()


def _own_append(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    cache = _own_cache(st, s)
    st.check(st.strata_kv_append(cache, s["k"], s["v"], s["T"], s["slots"], s["positions"], s["rope"],
                                 s["rope"].shape[0], c["rot"], q=s["q"], n_heads=c["Hq"], q_out=s["q_out"],
                                 k_stride=s["k"].stride(0), v_stride=s["v"].stride(0), q_stride=s["q"].stride(0),
                                 flags=st.STRATA_ROPE_NEIGHBOURS if c["neighbours"] else 0), "strata_kv_append")
    return {"q": s["q_out"], "k_codes": s["k_codes"], "v_codes": s["v_codes"], "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def _own_attention(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    cache = _own_cache(st, s)
    if "batch" not in s:
        s["batch"] = st.kv_batch(s["q_start"], s["kv_len"], s["table"], T=s["T"], max_q=s["max_q"], max_kv=s["max_kv"])
        n = st.strata_attention_workspace_size(cache, s["batch"], c["Hq"])
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    st.check(st.strata_attention_forward(cache, s["batch"], s["q"], c["Hq"], s["scale"], s["out"], s["ws"],
                                         s["ws"].numel(), window=c["window"], flags=st.STRATA_WS_REUSE),
             "strata_attention_forward")
    return s["out"]


def _plain_linear(s):
    c = s["case"]
    q = s["codes"]
    if c["bits"] == 4:  # two codes a byte, the even column in the low half, two's complement
        q = torch.stack([q & 15, q >> 4], -1).view(c["N"], c["K"]).float()
        q = torch.where(q > 7, q - 16, q)
    w = q.float().view(c["N"], -1, c["group"]) * s["scales"].float()[:, :, None]
    y = s["x"].float() @ w.view(c["N"], c["K"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _rotate(x, cos, sin, rot, neighbours):
    """x [T, H, D] in 32 or 64 bits, cos and sin [T, 1, rot/2]."""
    part, rest = x[..., :rot], x[..., rot:]
    if neighbours:
        a, b = part[..., 0::2], part[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([out, rest], -1)


def _scale_exp(absmax):
    """The smallest integer e with absmax * 2^-e <= 448, not below MIN_SCALE_EXP."""
    m, e = torch.frexp(absmax)  # m in [0.5, 1)
    e = torch.where(2 * m > E4M3_MAX_MANTISSA, e - 8, e - 9)
    return torch.where(absmax > 0, e.clamp_min(MIN_SCALE_EXP), torch.full_like(e, MIN_SCALE_EXP))


def _two_to(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_append(s):
    c = s["case"]
    T, Hq, Hkv, D, P, R = s["T"], c["Hq"], c["Hkv"], c["D"], c["page"], c["rot"]
    at = s["rope"][s["positions"].long()][:, None]
    cos, sin = at[..., :R // 2], at[..., R // 2:]
    q = _rotate(s["q"].float().view(T, Hq, D), cos, sin, R, c["neighbours"])
    k = _rotate(s["k"].float().view(T, Hkv, D), cos, sin, R, c["neighbours"])
    v = s["v"].float().view(T, Hkv, D)
    slots, pages = s["slots"].long(), s["pages"]
    of = torch.searchsorted(pages, slots // P)  # each row's place in the list of pages written to
    first = torch.full((len(pages),), P, device="cuda").index_reduce_(0, of, slots % P, "amin")
    for_old = torch.arange(P, device="cuda")[None] < first[:, None]  # the tokens that were there before
    out = {"q": q.to(torch.bfloat16).view(T, Hq * D)}
    out["k_codes"], out["k_scales"] = _plain_store(k, s["k_codes"], s["k_scales"], pages, of, slots % P, for_old)
    out["v_codes"], out["v_scales"] = _plain_store(v, s["v_codes"], s["v_scales"], pages, of, slots % P, for_old)
    return out


def _plain_store(x, codes, scales, pages, of, off, for_old):
    top = torch.zeros(len(pages), x.shape[1], device="cuda").index_reduce_(0, of, x.abs().amax(-1), "amax")
    need = _two_to(_scale_exp(top))
    before = torch.where(for_old[:, :1], scales[pages], torch.zeros_like(need))
    now = torch.maximum(need, before)
    kept = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    moved = (kept * (before / now)[:, :, None, None]).to(torch.float8_e4m3fn).float()
    block = torch.where(for_old[:, None, :, None], moved, kept)
    block[of, :, off] = x / now[of][:, :, None]
    codes.view(torch.uint8)[pages] = block.to(torch.float8_e4m3fn).view(torch.uint8)
    scales[pages] = now
    return codes, scales


def _plain_attention(s):
    c = s["case"]
    T, Hq, Hkv, D, P = s["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    B, Q, G = len(s["kv_len"]), s["max_q"], Hq // Hkv
    pages = s["table"].long()
    L = pages.shape[1] * P

    def gathered(codes, scales):  # [B, Hkv, L, D]
        x = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * scales[pages][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)

    row = s["q_start"][:-1, None].long() + torch.arange(Q, device="cuda")[None]
    real = torch.arange(Q, device="cuda")[None] < s["n_q"][:, None]
    q = s["q"].float()[row.clamp_max(T - 1)].view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    scores = (q @ gathered(s["k_codes"], s["k_scales"]).transpose(-1, -2)) * s["scale"]
    pos = (s["kv_len"] - s["n_q"])[:, None].long() + torch.arange(Q, device="cuda")[None]
    j = torch.arange(L, device="cuda")
    seen = (j <= pos[..., None]) & (j < s["kv_len"][:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    seen = seen[:, None, None].expand(B, 1, G, Q, L).reshape(B, 1, G * Q, L)
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    o = (p @ gathered(s["v_codes"], s["v_scales"])) / p.sum(-1, keepdim=True).clamp_min(1e-38)
    o = o.view(B, Hkv, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq * D)
    return o[real].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------- 64 bits

def _exact_e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), in 64 bits: steps of 2^-9 below 2^-6, else 3 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        N, K, G = case["N"], case["K"], case["group"]
        if case["bits"] == 4:
            byte = s["codes"].to(torch.int16)
            low, high = ((byte & 15) ^ 8) - 8, ((byte >> 4) ^ 8) - 8
            q = torch.empty(N, K, dtype=torch.float64, device="cuda")
            q[:, 0::2], q[:, 1::2] = low.double(), high.double()
        else:
            q = s["codes"].double()
        w = q * s["scales"].double().repeat_interleave(G, 1)
        y = s["x"].double() @ w.t()
        if s["bias"] is not None:
            y += s["bias"].double()
        if s["residual"] is not None:
            y += s["residual"].double()
        return y
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)


def _exact_append(case, s):
    Hq, Hkv, D, P, R = case["Hq"], case["Hkv"], case["D"], case["page"], case["rot"]
    T, h = s["T"], case["rot"] // 2
    at = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(at[:, :h], at[:, h:])[:, None]  # a rotation is a product of complex numbers

    def rotated(x, H):
        x = x.double().reshape(T, H, D)
        y = x.clone()
        if case["neighbours"]:
            z = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) * turn
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :h], x[..., h:R]) * turn
            y[..., :h], y[..., h:R] = z.real, z.imag
        return y

    out = {"q": rotated(s["q"], Hq).view(T, Hq * D)}
    off, page = s["slots"].long() % P, s["slots"].long() // P
    kinds = (("k_codes", "k_scales", rotated(s["k"], Hkv)), ("v_codes", "v_scales", s["v"].double().reshape(T, Hkv, D)))
    for name, scale_name, x in kinds:
        codes, scales = s[name].double(), s[scale_name].double()
        for p in s["pages"].tolist():
            rows = (page == p).nonzero()[:, 0]
            low = int(off[rows].min())
            top = x[rows].abs().amax((0, 2))
            m, e = torch.frexp(top / 448.0)  # m in [0.5, 1), exactly 0.5 for a power of two
            need = torch.exp2((e - (m == 0.5).int()).clamp_min(MIN_SCALE_EXP).double())
            now = torch.maximum(need, scales[p]) if low else need
            block = codes[p]
            block[:, :low] = _exact_e4m3(block[:, :low] * (scales[p] / now)[:, None, None])
            block[:, off[rows]] = _exact_e4m3(x[rows].transpose(0, 1) / now[:, None, None])
            scales[p] = now
        out[name], out[scale_name] = codes, scales
    return out


def _exact_attention(case, s):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros(s["T"], Hkv, Hq // Hkv, D, dtype=torch.float64, device="cuda")
    at = 0
    for b, (o, n) in enumerate(_lengths(case)):
        if n == 0:
            continue
        L = o + n
        pages = s["table"][b, :-(-L // case["page"])].long()
        for h in range(Hkv):
            k = (s["k_codes"][:, h][pages].double() * s["k_scales"][pages, h].double()[:, None, None]).view(-1, D)[:L]
            v = (s["v_codes"][:, h][pages].double() * s["v_scales"][pages, h].double()[:, None, None]).view(-1, D)[:L]
            q = s["q"][at:at + n].double().view(n, Hkv, Hq // Hkv, D)[:, h]
            t = torch.einsum("ngd,ld->ngl", q, k) * s["scale"]
            far = torch.arange(o, L, device="cuda")[:, None] - torch.arange(L, device="cuda")[None]
            hidden = far < 0
            if case["window"]:
                hidden |= far >= case["window"]
            t.masked_fill_(hidden[:, None], -math.inf)
            out[at:at + n, h] = torch.einsum("ngl,ld->ngd", torch.softmax(t, -1), v)
        at += n
    return out.view(s["T"], Hq * D)
