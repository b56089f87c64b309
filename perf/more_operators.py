"""Cases, plain forms and 64-bit definitions of what a serving process does with its paged 8-bit cache around the
attention: the append of normalised and rotated queries and keys, attention over a window and the first tokens
of a sequence, and the calls that share, extend, give back, move and copy pages.

Layer widths are those of the workload shapes in workloads/configs.py (hidden 1024, 4096, 5120, 7168); head
counts are the usual ones for such widths with 64- or 128-wide heads.
"""
import math

import torch

own = False

EPS = 1e-6            # added to the mean of squares
MIN_SCALE_EXP = -100  # a page's scale is 2^e with e at least this


# ---------------------------------------------------------------------------------------- cases

def listed():
    heads = {"Hq": 32, "Hkv": 8, "D": 128, "page": 64}
    return [
        # one new token for each of 16 sequences
        {"name": "append b16 q1", "op": "append", "n_seq": 16, "new": 1, "old": 2000, **heads, "rot": 128,
         "neighbours": False, "per_head": False},
        # short pieces on short contexts, 64-wide heads with weights of their own, half of each head rotated, small pages
        {"name": "append b7 ragged d64", "op": "append", "n_seq": 7, "new": 61, "old": 50, "Hq": 16, "Hkv": 4,
         "D": 64, "page": 16, "rot": 32, "neighbours": True, "per_head": True},
        # prompts entering the cache of a 7168-wide layer
        {"name": "append b3 prompts", "op": "append", "n_seq": 3, "new": 4096, "old": 100, "Hq": 56, "Hkv": 8,
         "D": 128, "page": 64, "rot": 128, "neighbours": False, "per_head": False},
        # one long conversation: the next token sees four first tokens and the last thousand
        {"name": "attention b1 q1 w1024", "op": "attention", "n_seq": 1, "new": 1, "len": 40000, **heads,
         "window": 1024, "sinks": 4, "ragged": False},
        # a decode batch of mixed lengths, a page of first tokens
        {"name": "attention b64 q1 w4096", "op": "attention", "n_seq": 64, "new": 1, "len": 16384, **heads,
         "window": 4096, "sinks": 64, "ragged": True},
        # pieces of prompts and single tokens in one batch, 64-wide heads, an empty sequence
        {"name": "attention b6 mixed w700", "op": "attention", "n_seq": 6, "new": 333, "len": 2500, "Hq": 28,
         "Hkv": 4, "D": 64, "page": 16, "window": 700, "sinks": 5, "ragged": True},
        # a piece of a long prompt
        {"name": "attention b1 q2048 w2048", "op": "attention", "n_seq": 1, "new": 2048, "len": 12288, **heads,
         "window": 2048, "sinks": 16, "ragged": False},
        # a prompt's old answers are dropped, 8 new ones start from it and take their first tokens, in one layer's cache
        {"name": "branch 1 to 8", "op": "branch", "parents": 1, "children": 8, "len": 1000, "new": 1, "Hkv": 8,
         "D": 128, "page": 64, "layers": 1, "pool": 256},
        # a server full of prompts with several answers each, pieces of several tokens, a few layers' caches
        {"name": "branch 48 to 5", "op": "branch", "parents": 48, "children": 5, "len": 6000, "new": 19, "Hkv": 4,
         "D": 128, "page": 64, "layers": 4, "pool": 16384},
        # few sequences move to a small pool
        {"name": "compact 5", "op": "compact", "n_seq": 5, "len": 700, "Hkv": 2, "D": 64, "page": 32, "layers": 2,
         "pool": 500},
        # a busy pool moves to another, among its sequences some that share their first pages
        {"name": "compact 60", "op": "compact", "n_seq": 60, "len": 8000, "Hkv": 8, "D": 128, "page": 64, "layers": 3,
         "pool": 12000},
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))
    return min(max(lo, hi), max(lo, v))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "branch", "compact"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    Hq = Hkv * rng.choice([1, 3, 4, 7, 8, 16] if Hkv < 8 else [1, 2, 4, 5])
    if op == "append":
        n_seq = _log_int(rng, 1, 40)
        return {"op": "append", "n_seq": n_seq, "new": _log_int(rng, 1, max(2, 8000 // n_seq)),
                "old": rng.choice([0, _log_int(rng, 1, 1500)]), "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
                "rot": rng.choice([D, D, D // 2, 0]), "neighbours": rng.random() < 0.3, "per_head": rng.random() < 0.3}
    if op == "attention":
        heads = {"Hq": Hq, "Hkv": Hkv, "D": D, "page": page}
        window, sinks = _log_int(rng, 1, 5000), _log_int(rng, 1, 300)
        if rng.random() < 0.6:  # single tokens, or a few
            n_seq = _log_int(rng, 1, 60)
            length = _log_int(rng, 16, 200000 // n_seq)
            return {"op": "attention", "n_seq": n_seq, "new": min(length, rng.choice([1, 1, 1, 2, 5])), "len": length,
                    **heads, "window": window, "sinks": sinks, "ragged": n_seq > 1}
        n_seq = _log_int(rng, 1, 6)
        length = _log_int(rng, 64, 8000 // n_seq)
        return {"op": "attention", "n_seq": n_seq, "new": _log_int(rng, 8, min(length, 1500)), "len": length, **heads,
                "window": window, "sinks": sinks, "ragged": n_seq > 1}
    if op == "branch":
        parents = _log_int(rng, 1, 60)
        children = rng.randint(1, 8)
        length = _log_int(rng, 5, 6000)
        new = _log_int(rng, 1, 70)
        need = parents * (-(-length // page) + children * (2 + -(-(new + page) // page)))
        return {"op": "branch", "parents": parents, "children": children, "len": length, "new": new, "Hkv": Hkv, "D": D,
                "page": page, "layers": rng.randint(1, 4), "pool": need + _log_int(rng, 1, 4000)}
    n_seq = _log_int(rng, 1, 60)
    length = _log_int(rng, 5, 200000 // n_seq)
    need = n_seq * -(-length // page)
    return {"op": "compact", "n_seq": n_seq, "len": length, "Hkv": Hkv, "D": D, "page": page,
            "layers": rng.randint(1, 4), "pool": need + _log_int(rng, 1, 4000)}


def _share(s):
    """A fixed spread of lengths: 1 for sequence 0, elevenths for the others."""
    return ((s * 7 + 3) % 11 + 1) / 11.0 if s else 1.0


def _lengths(case):
    """(tokens in the cache before, new tokens) of each sequence of an append or attention case."""
    rows = []
    for s in range(case["n_seq"]):
        if case["op"] == "append":
            rows.append((int(case["old"] * _share(s)), max(1, int(case["new"] * _share(s)))))
            continue
        part = _share(s) if case["ragged"] else 1.0
        total = max(1, int(case["len"] * part))
        if case["ragged"] and s == 2:    # one sequence has one new token,
            rows.append((total - 1, 1))
        elif case["ragged"] and s == 4:  # and one has no tokens at all in the cache
            rows.append((0, 0))
        else:
            new = min(total, max(1, int(case["new"] * part)))
            rows.append((total - new, new))
    return rows


def _pages(tokens, case):
    return -(-tokens // case["page"])


def _branches(case):
    """Of a branch case: parents' lengths, and each child's (parent, new tokens). Sequences are the parents, then the
    children, one of each parent after another."""
    lens = [max(1, int(case["len"] * _share(p))) for p in range(case["parents"])]
    kids = [(i % case["parents"], max(1, int(case["new"] * _share(i // case["parents"]))))
            for i in range(case["parents"] * case["children"])]
    return lens, kids


def _compact_rows(case):
    """Of a compact case: each sequence's length and how many of its first pages are sequence 0's."""
    rows = []
    for s in range(case["n_seq"]):
        n = max(1, int(case["len"] * _share(s)))
        rows.append((n, _pages(n, case) // 2 if s % 4 == 3 else 0))
    return rows


def _page_bytes(case):
    return case["Hkv"] * (2 * case["page"] * case["D"] + 8)


def work(case):
    if case["op"] == "append":
        rows = _lengths(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        T = sum(n for _, n in rows)
        # q in and out, k and v in, codes out, the table's rows, slots and positions, a scale pair a page
        pages = sum(_pages(o + n, case) - o // case["page"] for o, n in rows)
        return {"bytes": T * (4 * Hq * D + 6 * Hkv * D + 4 * case["rot"] + 8) + 8 * pages * Hkv,
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rot"]) + 4 * T * Hkv * D}
    if case["op"] == "attention":
        Hq, Hkv, D, W, S = case["Hq"], case["Hkv"], case["D"], case["window"], case["sinks"]
        kv = pairs = T = 0
        for o, n in _lengths(case):
            if n:
                first = max(0, o - W + 1)
                kv += o + n - first + min(first, S)
                pairs += sum(min(o + i + 1, W + min(S, max(0, o + i + 1 - W))) for i in range(n))
                T += n
        return {"bytes": kv * Hkv * 2 * D + 8 * (kv // case["page"]) * Hkv + 4 * T * Hq * D,
                "flops": 4 * pairs * Hq * D}
    if case["op"] == "branch":
        lens, kids = _branches(case)
        copies = sum(lens[p] % case["page"] != 0 for p, _ in kids)
        index = 4 * case["pool"] + sum(12 * _pages(lens[p] + n, case) + 8 * n for p, n in kids)
        return {"bytes": 2 * copies * case["layers"] * _page_bytes(case) + index, "flops": 0}
    rows = _compact_rows(case)
    live = sum(_pages(n, case) - shared for n, shared in rows)
    return {"bytes": 2 * live * case["layers"] * _page_bytes(case) + 8 * case["pool"] +
            sum(8 * _pages(n, case) for n, _ in rows), "flops": 0}


# ---------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev = {"device": "cuda", "generator": g}
    s = {"case": dict(case)}
    if case["op"] == "branch":
        return _prepare_branch(case, s, dev)
    if case["op"] == "compact":
        return _prepare_compact(case, s, dev)

    bf16 = torch.bfloat16
    rows = _lengths(case)
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["page"]
    B, T = len(rows), sum(n for _, n in rows)
    # pages that lie whole between the first tokens and the window of a sequence's first row have been given back
    held, width = [], max(1, max(_pages(o + n, case) for o, n in rows))
    for o, n in rows:
        hold = [True] * _pages(o + n, case)
        if case["op"] == "attention":
            for e in range(len(hold)):
                hold[e] = e * P < case["sinks"] or (e + 1) * P > o - case["window"] + 1
        held.append(hold + [False] * (width - len(hold)))
    hold = torch.tensor(held)
    n_pages = int(hold.sum()) + 3                                   # a few pages that no sequence holds
    order = torch.randperm(n_pages, **dev).to(torch.int32)          # a sequence's pages lie anywhere
    place = (torch.cumsum(hold.flatten().int(), 0) - 1).clamp_min(0).view(B, width).cuda()
    table = torch.where(hold.cuda(), order[place], -1).to(torch.int32).contiguous()
    old = torch.tensor([o for o, _ in rows], dtype=torch.int32, device="cuda")
    new = torch.tensor([n for _, n in rows], dtype=torch.int32, device="cuda")
    s["n_pages"] = n_pages
    _random_cache(s, n_pages, case, dev)
    s["table"], s["kv_len"], s["n_q"] = table, old + new, new
    start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.cumsum(new, 0)
    s["q_start"], s["T"] = start, T
    s["max_q"], s["max_kv"] = max(n for _, n in rows), max(o + n for o, n in rows)
    if case["op"] == "append":
        # each row's sequence and position, as a scheduler lists them
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), new.long(), output_size=T)
        pos = torch.arange(T, device="cuda") - start[seq].long() + old[seq].long()
        s["positions"] = pos.to(torch.int32)
        # q, k and v are column ranges of one projection's output, whose size differs from token to token
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, **dev) * torch.exp(torch.randn(T, 1, **dev) * 0.5)
        qkv = qkv.to(bf16)
        s["q"], s["k"], s["v"] = (qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:])
        s["q_weight"] = 1 + 0.3 * torch.randn(Hq if case["per_head"] else 1, D, **dev)
        s["k_weight"] = 1 + 0.3 * torch.randn(Hkv if case["per_head"] else 1, D, **dev)
        s["slots"] = (table[seq, pos // P].long() * P + pos % P).to(torch.int32)
        s["pages"] = torch.unique(s["slots"].long() // P)
        R = case["rot"]
        if R:
            freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
            ang = torch.arange(s["max_kv"], dtype=torch.float64, device="cuda")[:, None] * freq[None]
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["q_out"] = torch.empty(T, Hq * D, dtype=bf16, device="cuda")
    else:
        s["q"] = (torch.randn(T, Hq * D, **dev) * 1.5).to(bf16)
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.empty(T, Hq * D, dtype=bf16, device="cuda")
    return s


def _random_cache(s, n_pages, case, dev):
    """Codes and scales as an append leaves them."""
    shape = (n_pages, case["Hkv"], case["page"], case["D"])
    s["k_codes"] = (torch.randn(shape, **dev) * 70).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s["v_codes"] = (torch.randn(shape, **dev) * 70).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s["k_scales"] = torch.exp2(torch.randint(-7, -5, shape[:2], **dev).float())
    s["v_scales"] = torch.exp2(torch.randint(-8, -5, shape[:2], **dev).float())
    return s


def _count(table, n_pages):
    """How many entries name each page."""
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    return refs.scatter_add_(0, table.clamp_min(0).flatten().long(), (table >= 0).flatten().int())


def _prepare_branch(case, s, dev):
    lens, kids = _branches(case)
    P, n_pages, n_par = case["page"], case["pool"], len(lens)
    # before: parents hold pages anywhere in the pool, children the whole pages of their parents and one of their own
    order = torch.randperm(n_pages, **dev).tolist()
    width = max([_pages(n, case) for n in lens] + [_pages(lens[p] + n, case) for p, n in kids]) + 1
    table, length = [], []
    for n in lens:
        table.append([order.pop() for _ in range(_pages(n, case))])
        length.append(n)
    for i, (p, _) in enumerate(kids):
        whole = lens[p] // P
        table.append(table[p][:whole] + [order.pop()])
        length.append(whole * P + 1 + i % P)
    pad = [row + [-1] * (width - len(row)) for row in table]
    s["table"] = torch.tensor(pad, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    s["refs"] = _count(s["table"], n_pages)
    s["n_seq"], s["n_pages"], s["width"] = n_par + len(kids), n_pages, width
    s["parent"] = torch.tensor([-1] * n_par + [p for p, _ in kids], dtype=torch.int32, device="cuda")
    s["keep"] = torch.tensor([-1] * n_par + [0] * len(kids), dtype=torch.int32, device="cuda")
    s["new"] = torch.tensor([0] * n_par + [n for _, n in kids], dtype=torch.int32, device="cuda")
    s["T"] = sum(n for _, n in kids)
    s["n_moved"] = sum(lens[p] % P != 0 for p, _ in kids)
    for name, n in (("slots", s["T"]), ("positions", s["T"]), ("q_start", s["n_seq"] + 1), ("n_copies", 1)):
        s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["copies"] = torch.zeros(s["n_seq"], 2, dtype=torch.int32, device="cuda")
    s["caches"] = [_random_cache({}, n_pages, case, dev) for _ in range(case["layers"])]
    return s


def _prepare_compact(case, s, dev):
    rows = _compact_rows(case)
    n_pages = case["pool"]
    order = torch.randperm(n_pages, **dev).tolist()
    width = max(_pages(n, case) for n, _ in rows) + 1
    table = []
    for n, shared in rows:
        table.append(table[0][:shared] if shared else [])
        table[-1] = table[-1] + [order.pop() for _ in range(_pages(n, case) - shared)]
    live = n_pages - len(order)
    pad = [row + [-1] * (width - len(row)) for row in table]
    s["table"] = torch.tensor(pad, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor([n for n, _ in rows], dtype=torch.int32, device="cuda")
    s["refs"] = _count(s["table"], n_pages)
    s["n_seq"], s["n_pages"], s["width"], s["n_moved"] = len(rows), n_pages, width, live
    s["to_pages"] = live + 5  # the other pool is a little larger than what lives
    s["to_table"] = torch.zeros_like(s["table"])
    s["to_len"] = torch.zeros_like(s["kv_len"])
    s["to_refs"] = torch.zeros(s["to_pages"], dtype=torch.int32, device="cuda")
    s["copies"] = torch.zeros(s["to_pages"], 2, dtype=torch.int32, device="cuda")
    s["n_copies"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["caches"] = [_random_cache({}, n_pages, case, dev) for _ in range(case["layers"])]
    s["to_caches"] = [{k: torch.zeros((s["to_pages"],) + v.shape[1:], dtype=v.dtype, device="cuda")
                       for k, v in c.items()} for c in s["caches"]]
    return s


# ---------------------------------------------------------------------------------------- passes

def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "branch": _own_branch,
                "compact": _own_compact}[op](s)
    return {"append": _plain_append, "attention": _plain_attention, "branch": _plain_branch,
            "compact": _plain_compact}[op](s)


def _own_cache(st, s, n_pages, case):
    return st.PagedKVCache(n_pages, case["Hkv"], case["D"], case["page"], k_codes=s["k_codes"], v_codes=s["v_codes"],
                           k_scales=s["k_scales"], v_scales=s["v_scales"])


def _own_append(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    if "cache" not in s:
        s["cache"] = _own_cache(st, s, s["n_pages"], c)
        s["norm"] = st.QKNorm(s["q_weight"], s["k_weight"], c["D"], eps=EPS)
    rope = s.get("rope")
    st.check(st.strata_kv_append_normed(s["cache"].struct(), s["norm"].struct(), s["k"], s["v"], s["T"], s["slots"],
                                        s["positions"], rope, 0 if rope is None else rope.shape[0], c["rot"], q=s["q"],
                                        n_heads=c["Hq"], q_out=s["q_out"], k_stride=s["k"].stride(0),
                                        v_stride=s["v"].stride(0), q_stride=s["q"].stride(0),
                                        flags=st.STRATA_ROPE_NEIGHBOURS if c["neighbours"] else 0),
             "strata_kv_append_normed")
    return {"q": s["q_out"], "k_codes": s["k_codes"], "v_codes": s["v_codes"], "k_scales": s["k_scales"],
            "v_scales": s["v_scales"]}


def _own_attention(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    if "cache" not in s:
        s["cache"] = _own_cache(st, s, s["n_pages"], c)
        s["batch"] = st.kv_batch(s["q_start"], s["kv_len"], s["table"], T=s["T"], max_q=s["max_q"], max_kv=s["max_kv"])
        n = st.strata_attention_workspace_size(s["cache"].struct(), s["batch"], c["Hq"])
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    st.check(st.strata_attention_sinks_forward(s["cache"].struct(), s["batch"], s["q"], c["Hq"], s["scale"], s["out"],
                                               s["ws"], s["ws"].numel(), window=c["window"], n_sinks=c["sinks"],
                                               flags=st.STRATA_WS_REUSE), "strata_attention_sinks_forward")
    return s["out"]


def _own_branch(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    if "pages" not in s:
        s["pages"] = st.PageTable(s["n_pages"], s["n_seq"], s["width"], c["page"], page_table=s["table"],
                                  kv_len=s["kv_len"], refs=s["refs"])
        s["layers"] = st.cache_array([_own_cache(st, x, s["n_pages"], c) for x in s["caches"]])
    pages = s["pages"].struct()
    st.check(st.strata_kv_pages_release(pages, s["keep"]), "strata_kv_pages_release")
    st.check(st.strata_kv_pages_fork(pages, s["parent"]), "strata_kv_pages_fork")
    st.check(st.strata_kv_pages_extend(pages, s["new"], s["T"], s["slots"], s["positions"], s["q_start"], s["copies"],
                                       s["n_copies"]), "strata_kv_pages_extend")
    st.check(st.strata_kv_copy_pages(s["layers"], s["layers"], s["copies"], s["n_copies"], s["n_seq"]),
             "strata_kv_copy_pages")
    return _branch_outputs(s)


def _branch_outputs(s):
    return {"table": s["table"], "kv_len": s["kv_len"], "refs": s["refs"], "slots": s["slots"],
            "positions": s["positions"], "q_start": s["q_start"], "copies": s["copies"], "n_copies": s["n_copies"],
            "caches": s["caches"]}


def _own_compact(s):
    import int4_grouped_expert_gb300 as st
    c = s["case"]
    if "from" not in s:
        s["from"] = st.PageTable(s["n_pages"], s["n_seq"], s["width"], c["page"], page_table=s["table"],
                                 kv_len=s["kv_len"], refs=s["refs"])
        s["to"] = st.PageTable(s["to_pages"], s["n_seq"], s["width"], c["page"], page_table=s["to_table"],
                               kv_len=s["to_len"], refs=s["to_refs"])
        s["src"] = st.cache_array([_own_cache(st, x, s["n_pages"], c) for x in s["caches"]])
        s["dst"] = st.cache_array([_own_cache(st, x, s["to_pages"], c) for x in s["to_caches"]])
        n = st.strata_kv_pages_compact_workspace_size(s["from"].struct())
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    st.check(st.strata_kv_pages_compact(s["from"].struct(), s["to"].struct(), s["copies"], s["n_copies"], s["ws"],
                                        s["ws"].numel()), "strata_kv_pages_compact")
    st.check(st.strata_kv_copy_pages(s["src"], s["dst"], s["copies"], s["n_copies"], s["to_pages"]),
             "strata_kv_copy_pages")
    return _compact_outputs(s)


def _compact_outputs(s):
    return {"table": s["to_table"], "kv_len": s["to_len"], "refs": s["to_refs"], "copies": s["copies"],
            "n_copies": s["n_copies"], "caches": s["to_caches"]}


def _normed(x, w):
    """x [T, H, D] in 32 bits, w [H or 1, D]."""
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _rotate(x, cos, sin, rot, neighbours):
    """x [T, H, D], cos and sin [T, 1, rot/2]."""
    part, rest = x[..., :rot], x[..., rot:]
    if neighbours:
        a, b = part[..., 0::2], part[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([out, rest], -1)


def _scale_of(absmax):
    """2^e with the smallest integer e that has absmax <= 448 * 2^e, not below MIN_SCALE_EXP."""
    m, e = torch.frexp(absmax)  # m in [0.5, 1); 448 is 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(absmax > 0, e.clamp_min(MIN_SCALE_EXP), torch.full_like(e, MIN_SCALE_EXP))
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_append(s):
    c = s["case"]
    T, Hq, Hkv, D, P, R = s["T"], c["Hq"], c["Hkv"], c["D"], c["page"], c["rot"]
    q = _normed(s["q"].float().view(T, Hq, D), s["q_weight"])
    k = _normed(s["k"].float().view(T, Hkv, D), s["k_weight"])
    v = s["v"].float().view(T, Hkv, D)
    if R:
        at = s["rope"][s["positions"].long()][:, None]
        cos, sin = at[..., :R // 2], at[..., R // 2:]
        q, k = _rotate(q, cos, sin, R, c["neighbours"]), _rotate(k, cos, sin, R, c["neighbours"])
    slots, pages = s["slots"].long(), s["pages"]
    of = torch.searchsorted(pages, slots // P)  # each row's place in the list of pages written to
    first = torch.full((len(pages),), P, device="cuda").index_reduce_(0, of, slots % P, "amin")
    before = torch.arange(P, device="cuda")[None] < first[:, None]  # the tokens that were there
    out = {"q": q.to(torch.bfloat16).view(T, Hq * D)}
    for name, x in (("k", k), ("v", v)):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        top = torch.zeros(len(pages), Hkv, device="cuda").index_reduce_(0, of, x.abs().amax(-1), "amax")
        need = _scale_of(top)
        was = torch.where(before[:, :1], scales[pages], torch.zeros_like(need))
        now = torch.maximum(need, was)
        kept = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        block = torch.where(before[:, None, :, None], kept * (was / now)[:, :, None, None], kept)
        block[of, :, slots % P] = x / now[of][:, :, None]
        codes.view(torch.uint8)[pages] = block.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[pages] = now
        out[name + "_codes"], out[name + "_scales"] = codes, scales
    return out


def _plain_attention(s):
    c = s["case"]
    T, Hq, Hkv, D, P = s["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    B, Q, G = len(s["kv_len"]), s["max_q"], Hq // Hkv
    pages = s["table"].long().clamp_min(0)
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
    seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    seen = seen[:, None, None].expand(B, 1, G, Q, L).reshape(B, 1, G * Q, L)
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    o = (p @ gathered(s["v_codes"], s["v_scales"])) / p.sum(-1, keepdim=True).clamp_min(1e-38)
    o = o.view(B, Hkv, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq * D)
    return o[real].to(torch.bfloat16)


def _plain_branch(s):
    c, P = s["case"], s["case"]["page"]
    table, refs = s["table"], s["refs"]
    entry = torch.arange(s["width"], dtype=torch.int32, device="cuda")[None]

    def pages_of(tokens):
        return (tokens + (P - 1)) // P

    # the children let go of what they hold
    length = torch.where(s["keep"] >= 0, torch.minimum(s["keep"], s["kv_len"]), s["kv_len"])
    gone = (entry >= pages_of(length)[:, None]) & (table >= 0)
    refs.scatter_add_(0, table.clamp_min(0).flatten().long(), -gone.flatten().int())
    table.masked_fill_(gone, -1)
    # and take their parents' pages
    child = s["parent"] >= 0
    of = s["parent"].clamp_min(0).long()
    length = torch.where(child, length[of], length)
    table.copy_(torch.where(child[:, None], table[of], table))
    taken = child[:, None] & (table >= 0)
    refs.scatter_add_(0, table.clamp_min(0).flatten().long(), taken.flatten().int())
    # room for the new tokens; an unfinished page that others hold too is left to them
    new = s["new"]
    last = table.gather(1, (length // P)[:, None].long())[:, 0]
    moved = (length % P != 0) & (new > 0) & (refs[last.clamp_min(0).long()] > 1)
    first = torch.where(moved, length // P, pages_of(length))
    end = pages_of(length + new)
    need = torch.where(new > 0, end - first, torch.zeros_like(end))
    at = torch.cumsum(need, 0) - need
    free = refs == 0
    rank = torch.where(free, torch.cumsum(free, 0) - 1, s["n_pages"])
    lowest = torch.zeros(s["n_pages"] + 1, dtype=torch.int32, device="cuda")
    lowest.scatter_(0, rank, torch.arange(s["n_pages"], dtype=torch.int32, device="cuda"))
    mine = (entry >= first[:, None]) & (entry < (first + need)[:, None])
    given = lowest[torch.where(mine, at[:, None] + entry - first[:, None], 0).long()]
    refs.scatter_add_(0, last.clamp_min(0).long(), -moved.int())
    refs.scatter_add_(0, given.flatten().long(), mine.flatten().int())
    copy_at = torch.where(moved, torch.cumsum(moved, 0) - 1, s["n_seq"])
    copies = torch.zeros(s["n_seq"] + 1, 2, dtype=torch.int32, device="cuda")
    pairs = torch.stack([last, lowest[at.clamp_max(s["n_pages"]).long()]], 1)
    copies[copy_at] = pairs.int()
    s["copies"][:s["n_moved"]] = copies[:s["n_moved"]]
    s["n_copies"].copy_(moved.sum().int())
    table.copy_(torch.where(mine, given, table))
    s["q_start"][1:] = torch.cumsum(new, 0)
    seq = torch.repeat_interleave(torch.arange(s["n_seq"], device="cuda"), new.long(), output_size=s["T"])
    pos = length[seq] + torch.arange(s["T"], device="cuda") - s["q_start"][seq]
    s["positions"].copy_(pos)
    s["slots"].copy_(table[seq, pos.long() // P] * P + pos % P)
    s["kv_len"].copy_(length + new)
    _plain_copy(s["caches"], s["caches"], s["copies"][:s["n_moved"]])
    return _branch_outputs(s)


def _plain_copy(src, dst, pairs):
    a, b = pairs[:, 0].long(), pairs[:, 1].long()
    for x, y in zip(src, dst):
        for name in x:
            kind = torch.uint8 if x[name].dtype == torch.float8_e4m3fn else x[name].dtype
            y[name].view(kind)[b] = x[name].view(kind)[a]


def _plain_compact(s):
    P = s["case"]["page"]
    live = s["refs"] > 0
    rank = torch.cumsum(live, 0, dtype=torch.int32) - 1
    entry = torch.arange(s["width"], dtype=torch.int32, device="cuda")[None]
    held = (entry < ((s["kv_len"] + (P - 1)) // P)[:, None]) & (s["table"] >= 0)
    s["to_table"].copy_(torch.where(held, rank[s["table"].clamp_min(0).long()], -1))
    s["to_len"].copy_(s["kv_len"])
    to = torch.where(live, rank, s["to_pages"]).long()
    counts = torch.zeros(s["to_pages"] + 1, dtype=torch.int32, device="cuda").scatter_(0, to, s["refs"])
    counts[s["to_pages"]] = 0
    s["to_refs"].copy_(counts[:s["to_pages"]])
    pairs = torch.zeros(s["to_pages"] + 1, 2, dtype=torch.int32, device="cuda")
    pairs[to] = torch.stack([torch.arange(s["n_pages"], dtype=torch.int32, device="cuda"), rank], 1)
    s["copies"][:s["n_moved"]] = pairs[:s["n_moved"]]
    s["n_copies"].copy_(live.sum().int())
    _plain_copy(s["caches"], s["to_caches"], s["copies"][:s["n_moved"]])
    return _compact_outputs(s)


# ---------------------------------------------------------------------------------------- 64 bits

def _exact_e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even), in 64 bits: steps of 2^-9 below 2^-6, else 3 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "branch": _exact_branch,
            "compact": _exact_compact}[case["op"]](case, s)


def _exact_append(case, s):
    Hq, Hkv, D, P, R = case["Hq"], case["Hkv"], case["D"], case["page"], case["rot"]
    T, h = s["T"], case["rot"] // 2

    def turned(x, weight, H):
        x = x.double().reshape(T, H, D)
        size = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + EPS)
        y = x / size * weight.double()
        if R == 0:
            return y
        at = s["rope"].double()[s["positions"].long()]
        turn = torch.complex(at[:, :h], at[:, h:])[:, None]  # a rotation is a product of complex numbers
        out = y.clone()
        if case["neighbours"]:
            z = torch.complex(y[..., 0:R:2], y[..., 1:R:2]) * turn
            out[..., 0:R:2], out[..., 1:R:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :h], y[..., h:R]) * turn
            out[..., :h], out[..., h:R] = z.real, z.imag
        return out

    out = {"q": turned(s["q"], s["q_weight"], Hq).view(T, Hq * D)}
    off, page = s["slots"].long() % P, s["slots"].long() // P
    kinds = (("k_codes", "k_scales", turned(s["k"], s["k_weight"], Hkv)),
             ("v_codes", "v_scales", s["v"].double().reshape(T, Hkv, D)))
    for name, scale_name, x in kinds:
        codes, scales = s[name].double(), s[scale_name].double()
        for p in s["pages"].tolist():
            rows = (page == p).nonzero()[:, 0]
            low = int(off[rows].min())
            m, e = torch.frexp(x[rows].abs().amax((0, 2)) / 448.0)  # m in [0.5, 1), exactly 0.5 for a power of two
            need = torch.exp2((e - (m == 0.5).int()).clamp_min(MIN_SCALE_EXP).double())
            now = torch.maximum(need, scales[p]) if low else need
            block = codes[p]
            block[:, :low] = _exact_e4m3(block[:, :low] * (scales[p] / now)[:, None, None])
            block[:, off[rows]] = _exact_e4m3(x[rows].transpose(0, 1) / now[:, None, None])
            scales[p] = now
        out[name], out[scale_name] = codes, scales
    return out


def _exact_attention(case, s):
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["page"]
    out = torch.zeros(s["T"], Hkv, Hq // Hkv, D, dtype=torch.float64, device="cuda")
    at = 0
    for b, (o, n) in enumerate(_lengths(case)):
        if n == 0:
            continue
        # the tokens that any row sees, by their positions
        first = max(0, o - case["window"] + 1)
        tok = torch.cat([torch.arange(min(first, case["sinks"])), torch.arange(first, o + n)]).cuda()
        page, off = s["table"][b].long()[tok // P], tok % P
        far = torch.arange(o, o + n, device="cuda")[:, None] - tok[None]
        hidden = (far < 0) | ((far >= case["window"]) & (tok[None] >= case["sinks"]))
        for h in range(Hkv):
            k = s["k_codes"].view(torch.uint8)[page, h, off].view(torch.float8_e4m3fn).double()
            v = s["v_codes"].view(torch.uint8)[page, h, off].view(torch.float8_e4m3fn).double()
            k, v = k * s["k_scales"][page, h].double()[:, None], v * s["v_scales"][page, h].double()[:, None]
            q = s["q"][at:at + n].double().view(n, Hkv, Hq // Hkv, D)[:, h]
            t = torch.einsum("ngd,ld->ngl", q, k) * s["scale"]
            t.masked_fill_(hidden[:, None], -math.inf)
            out[at:at + n, h] = torch.einsum("ngl,ld->ngd", torch.softmax(t, -1), v)
        at += n
    return out.view(s["T"], Hq * D)


def _ints(rows):
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _exact_branch(case, s):
    """The same calls on host lists, one sequence after another."""
    P = case["page"]
    table = [row[:row.index(-1)] if -1 in row else row for row in s["table"].tolist()]
    length, refs, new = s["kv_len"].tolist(), s["refs"].tolist(), s["new"].tolist()
    kids = [(c, p) for c, p in enumerate(s["parent"].tolist()) if p >= 0]
    for c, _ in kids:
        for page in table[c]:
            refs[page] -= 1
        table[c], length[c] = [], 0
    for c, p in kids:
        table[c], length[c] = list(table[p]), length[p]
        for page in table[c]:
            refs[page] += 1
    free = iter([page for page, n in enumerate(refs) if n == 0])
    before = list(refs)
    slots, positions, q_start, copies = [], [], [0], []
    for row, n in enumerate(new):
        if n and length[row] % P and before[table[row][-1]] > 1:
            page = next(free)
            copies.append([table[row][-1], page])
            refs[table[row][-1]] -= 1
            refs[page] = 1
            table[row][-1] = page
        for _ in range(n):
            if length[row] == len(table[row]) * P:
                table[row].append(next(free))
                refs[table[row][-1]] = 1
            slots.append(table[row][length[row] // P] * P + length[row] % P)
            positions.append(length[row])
            length[row] += 1
        q_start.append(len(slots))
    caches = [{k: v.clone() for k, v in c.items()} for c in s["caches"]]
    for c, was in zip(caches, s["caches"]):
        for a, b in copies:
            for k in c:
                c[k].view(torch.uint8)[b] = was[k].view(torch.uint8)[a]
    full = [row + [-1] * (s["width"] - len(row)) for row in table]
    return {"table": _ints(full), "kv_len": _ints(length), "refs": _ints(refs), "slots": _ints(slots),
            "positions": _ints(positions), "q_start": _ints(q_start),
            "copies": _ints(copies + [[0, 0]] * (s["n_seq"] - len(copies))), "n_copies": _ints([len(copies)]),
            "caches": [{k: v.double() for k, v in c.items()} for c in caches]}


def _exact_compact(case, s):
    refs, n = s["refs"].tolist(), s["to_pages"]
    live = [page for page, count in enumerate(refs) if count > 0]
    where = {page: i for i, page in enumerate(live)}
    table = [[where.get(page, -1) for page in row] for row in s["table"].tolist()]
    index = _ints(live)
    caches = []
    for c in s["caches"]:
        caches.append({})
        for k, v in c.items():
            kind = v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v
            full = torch.zeros((n,) + v.shape[1:], dtype=torch.float64, device="cuda")
            full[:len(live)] = torch.index_select(kind, 0, index).view(v.dtype).double()
            caches[-1][k] = full
    pad = n - len(live)
    return {"table": _ints(table), "kv_len": _ints(s["kv_len"].tolist()),
            "refs": _ints([refs[page] for page in live] + [0] * pad),
            "copies": _ints([[page, i] for i, page in enumerate(live)] + [[0, 0]] * pad), "n_copies": _ints([len(live)]),
            "caches": caches}
