"""Operators that decide what a paged CSA2 cache keeps: what is measured, and their plain forms.

* weigh   csa2_attn_weight: the attention weight that every cache entry has got from
          a step's queries, summed over queries and heads and added to a running sum;
* evict   csa2_evict: the entries of largest accumulated weight, and the latest ones,
          moved together at the front of a sequence's pages (here: into other pages,
          so that a pass finds what the one before found);
* verify  csa2_verify_drafts: which drafted tokens the target model's probabilities
          accept, from given random numbers, and the token that comes after them.

`own` False: elementary torch operations, in 32 bits (64 where 32 lose what
matters), rounded once at the end.  `own` True: the library's entry points.
"""
import math

import torch

own = False

H, D, KV_BYTES = 64, 512, 288
SCALE = 1.0 / math.sqrt(512.0)
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding sequence of the 4,096-entry workload: latency
        {"name": "weigh_1x4096", "op": "weigh", "n_seq": 1, "queries": 1, "n": 4096, "sel": 0, "page": 64, "ragged": False},
        # five draft positions of 8 sequences, over the 512 entries that each of them selected
        {"name": "weigh_sel_40x512", "op": "weigh", "n_seq": 8, "queries": 5, "n": 65536, "sel": 512, "page": 64,
         "ragged": False},
        # the last 32 queries of four prompts of unequal, odd lengths vote before their caches are cut down
        {"name": "weigh_votes_4x32", "op": "weigh", "n_seq": 4, "queries": 32, "n": 40_001, "sel": 0, "page": 48,
         "ragged": True},
        # five draft positions of each of the 32 x 65,536 decode workload's sequences, dense
        {"name": "weigh_drafts_32x65536", "op": "weigh", "n_seq": 32, "queries": 5, "n": 65536, "sel": 0, "page": 64,
         "ragged": False},
        # a token of each of the 8 x 1,048,576 long-context workload's sequences, dense
        {"name": "weigh_8x1M", "op": "weigh", "n_seq": 8, "queries": 1, "n": 1 << 20, "sel": 0, "page": 128,
         "ragged": False},
        # one sequence cut down to half: latency
        {"name": "evict_1x4096", "op": "evict", "n_seq": 1, "n": 4096, "keep": 2048, "recent": 128, "page": 64, "ragged": False},
        # a served batch of unequal lengths, a budget that some are below, pages that do not divide anything
        {"name": "evict_ragged_33", "op": "evict", "n_seq": 33, "n": 40_001, "keep": 9_999, "recent": 300, "page": 48,
         "ragged": True},
        # the long-context workload cut down to half
        {"name": "evict_8x1M", "op": "evict", "n_seq": 8, "n": 1 << 20, "keep": 1 << 19, "recent": 4096, "page": 128,
         "ragged": False},
        # five drafts of one sequence: latency
        {"name": "verify_1", "op": "verify", "mode": "sample", "n_seq": 1, "drafts": 5, "vocab": 131072, "type": "f32",
         "draft_probs": True, "ragged": False},
        # a batch of drafting sequences, of unequal draft counts, over an odd vocabulary in 16 bits
        {"name": "verify_64_bf16", "op": "verify", "mode": "sample", "n_seq": 64, "drafts": 5, "vocab": 100_003,
         "type": "bf16", "draft_probs": True, "ragged": True},
        # many sequences, drafts from a lookup (no draft probabilities)
        {"name": "verify_256_lookup", "op": "verify", "mode": "sample", "n_seq": 256, "drafts": 3, "vocab": 131072,
         "type": "f32", "draft_probs": False, "ragged": False},
        # greedy decoding of the same batch: the target's logits
        {"name": "verify_64_greedy", "op": "verify", "mode": "greedy", "n_seq": 64, "drafts": 5, "vocab": 131072,
         "type": "bf16", "draft_probs": False, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["weigh", "weigh", "evict", "verify"])
    page = rng.choice([16, 32, 48, 64, 100, 128])
    if op == "weigh":
        n_seq, queries = _log(rng, 1, 40), rng.choice([1, 1, 2, 5, 6, _log(rng, 3, 48)])
        n = min(_log(rng, 1, 1 << 20), 4_000_000 // (n_seq * queries))
        return {"op": op, "n_seq": n_seq, "queries": queries, "n": max(n, queries),
                "sel": rng.choice([0, 0, 512, rng.randint(1, 512)]), "page": page, "ragged": rng.random() < 0.5}
    if op == "evict":
        n_seq = _log(rng, 1, 200)
        n = min(_log(rng, 1, 1 << 20), 4_000_000 // n_seq)
        keep = max(1, int(n * rng.uniform(0.05, 1.05)))
        return {"op": op, "n_seq": n_seq, "n": n, "keep": keep, "recent": rng.choice([0, 1, 128, rng.randint(0, keep)]),
                "page": page, "ragged": rng.random() < 0.5}
    mode = rng.choice(["sample", "sample", "greedy"])
    vocab = _log(rng, 1000, 150_000)
    drafts = rng.choice([0, 1, 2, 3, 5, 8])
    n_seq = max(1, min(_log(rng, 1, 400), 20_000_000 // (vocab * (drafts + 1))))
    return {"op": op, "mode": mode, "n_seq": n_seq, "drafts": drafts, "vocab": vocab,
            "type": rng.choice(["f32", "bf16", "f16"]), "draft_probs": mode == "sample" and rng.random() < 0.7,
            "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------ shapes that follow from a case
def _mix(i):
    """A fixed spread of i over [0, 1)."""
    return (i * 2654435761 + 40503) % (1 << 32) / float(1 << 32)


def _lens(c, least=1):
    """Entries of every sequence; the first is always the longest."""
    n = c["n"]
    return [n if i == 0 or not c["ragged"] else max(least, int(n * _mix(i))) for i in range(c["n_seq"])]


def _queries(c):
    """(sequence, visible entries) of every query, in sequence order: query t of G sees up to itself."""
    g = c["queries"]
    return [(s, max(1, n - g + t + 1)) for s, n in enumerate(_lens(c, g)) for t in range(g)]


def _kept(c):
    return [min(n, c["keep"]) for n in _lens(c)]


def _rows(c):
    """Tokens of the step of every sequence: the last sampled one and its drafts."""
    g = c["drafts"]
    return [1 + (int(_mix(i + 5) * (g + 1)) if c["ragged"] and i > 0 else g) for i in range(c["n_seq"])]


def _agree(c):
    """Drafts that the greedy target agrees with, of every sequence."""
    return [min(r - 1, int(_mix(i + 31) * (r + 1))) for i, r in enumerate(_rows(c))]


def work(case):
    if case["op"] == "weigh":
        qs = _queries(case)
        k = case["sel"]
        pairs = sum(min(k, v) if k else v for _, v in qs)
        if k:                                   # selections of one sequence: any of their entries may be the same
            entries = sum(max(min(k, v) for s, v in qs if s == b) for b in range(case["n_seq"]))
        else:
            entries = sum(_lens(case, case["queries"]))
        return {"bytes": entries * (KV_BYTES + 8) + len(qs) * (2 * H * D + 4 * H), "flops": 2.0 * H * D * pairs}
    if case["op"] == "evict":
        kept = sum(_kept(case))
        return {"bytes": 4 * sum(_lens(case)) + kept * (2 * KV_BYTES + 4 + 4), "flops": 0}
    size = 4 if case["type"] == "f32" else 2
    if case["mode"] == "greedy":                # the rows up to the first refusal
        return {"bytes": size * case["vocab"] * sum(a + 1 for a in _agree(case)), "flops": 0}
    return {"bytes": size * case["vocab"] * case["n_seq"], "flops": 0}


# ------------------------------------------------------------------ record formats, elementary
def _e2m1_pairs():
    """[256, 2]: the two FP4 values of a byte, low nibble first."""
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    val = mag + [-m for m in mag]
    return torch.tensor([[val[b & 15], val[b >> 4]] for b in range(256)], dtype=torch.float32, device=DEV)


def _kv_values(rec, pairs):
    """[n, 288] record bytes -> [n, 512] fp32 latents."""
    v = pairs.index_select(0, rec[:, :256].reshape(-1).to(torch.int32)).view(-1, 32, 16)
    s = rec[:, 256:].contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    return (v * s[:, :, None]).view(-1, D)


def _pack_kv(x):
    """fp32 [n, 512] -> record bytes [n, 288]: one E4M3 scale for 16 channels, FP4 codes to the nearest."""
    g = x.view(-1, 32, 16)
    s8 = (g.abs().amax(2) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = g / s8.to(torch.float32).clamp(min=2.0 ** -9)[:, :, None]
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(y.abs(), edge, out_int32=True) + 8 * torch.signbit(y).to(torch.int32)
    code = code.view(-1, 256, 2)
    return torch.cat([(code[:, :, 0] | (code[:, :, 1] << 4)).to(torch.uint8), s8.view(torch.uint8)], 1)


# ------------------------------------------------------------------ states
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _records(g, n):
    out = torch.empty((n, KV_BYTES), dtype=torch.uint8, device=DEV)
    for a in range(0, n, 1 << 18):
        b = min(n, a + (1 << 18))
        out[a:b] = _pack_kv(torch.randn((b - a, D), generator=g, device=DEV))
    return out


def _tables(g, lens, p):
    """Pages of sequences of these lengths in random order: (table, pages in all)."""
    pages = [-(-n // p) for n in lens]
    n_pages, cols = sum(pages) + 3, max(pages)
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    have = _i32(pages)
    first = torch.cumsum(have, 0) - have
    col = torch.arange(cols, device=DEV, dtype=torch.int32)
    table = torch.where(col < have[:, None], perm[(first[:, None] + col).clamp(max=n_pages - 1).long()],
                        torch.full((), -1, dtype=torch.int32, device=DEV))
    return table.contiguous(), n_pages


def prepare(case, seed):
    return {"weigh": _prepare_weigh, "evict": _prepare_evict, "verify": _prepare_verify}[case["op"]](case, seed)


def _prepare_weigh(c, seed):
    g = _gen(seed)
    p, lens, qs = c["page"], _lens(c, c["queries"]), _queries(c)
    nq = len(qs)
    table, n_pages = _tables(g, lens, p)
    vis = _i32([v for _, v in qs])
    seen = vis.clamp(max=c["sel"]) if c["sel"] else vis
    s = {"op": "weigh", "page": p, "n_pages": n_pages, "n_seq": c["n_seq"], "n_q": nq, "lens": lens, "queries": c["queries"],
         "table": table, "pages": _records(g, n_pages * p).view(n_pages, p, KV_BYTES),
         "q": torch.randn((nq, H, D), generator=g, device=DEV).bfloat16(),
         "first": _i32([b * c["queries"] for b in range(c["n_seq"] + 1)]), "n_vis": vis, "sel": None,
         # about what these queries' attention returns: logits of unit size over what they see and the window
         "lse": torch.log(seen.float() + 128.0)[:, None] + 0.5 + 0.1 * torch.randn((nq, H), generator=g, device=DEV),
         "decay": 0.875,
         # what a few such steps before have left: 64 heads' weights, unequally over the entries
         "prior": torch.exp(1.5 * torch.randn(n_pages * p, generator=g, device=DEV)) * (H * c["queries"] / c["n"]),
         "weight": torch.zeros(n_pages * p, dtype=torch.float32, device=DEV)}
    if c["sel"]:
        # distinct visible entries in ascending order, -1 behind them: one of each of `sel` equal parts of the row
        k = c["sel"]
        u = torch.rand((nq, k), generator=g, device=DEV, dtype=torch.float64)
        a = torch.arange(k, device=DEV, dtype=torch.float64)
        v = vis.double()[:, None]
        lo, hi = (a * v / k).ceil(), ((a + 1) * v / k).ceil() - 1
        long_row = torch.minimum(torch.maximum(((a + u) * v / k).floor(), lo), hi)
        short_row = torch.where(a < v, a, torch.full((), -1.0, dtype=torch.float64, device=DEV))
        s["sel"] = torch.where(v >= k, long_row, short_row).to(torch.int32).contiguous()
    if own:
        import compressed_sparse_attention_index_gb300 as lib
        s["ws"] = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, nq, c["n_seq"], c["sel"]),
                              dtype=torch.uint8, device=DEV)
    return s


def _prepare_evict(c, seed):
    g = _gen(seed)
    p, lens, kept = c["page"], _lens(c), _kept(c)
    table, n_pages = _tables(g, lens, p)
    dst_table, n_dst = _tables(g, kept, p)
    n = n_pages * p
    # accumulated weights: most entries have got little, and one in a hundred nothing yet
    w = torch.exp(2.0 * torch.randn(n, generator=g, device=DEV) - 8.0)
    w = torch.where(torch.rand(n, generator=g, device=DEV) < 0.01, torch.zeros((), device=DEV), w)
    s = {"op": "evict", "page": p, "n_pages": n_pages, "n_dst": n_dst, "n_seq": c["n_seq"], "lens": lens, "kept": kept,
         "recent": c["recent"], "table": table, "dst_table": dst_table, "weight": w,
         "pages": _records(g, n).view(n_pages, p, KV_BYTES),
         "seq_len": _i32(lens), "keep": _i32([c["keep"]] * c["n_seq"]),
         "dst_pages": torch.zeros((n_dst, p, KV_BYTES), dtype=torch.uint8, device=DEV),
         "dst_weight": torch.zeros(n_dst * p, dtype=torch.float32, device=DEV),
         "new_len": torch.empty(c["n_seq"], dtype=torch.int32, device=DEV),
         "from": torch.full((c["n_seq"], max(kept)), -1, dtype=torch.int32, device=DEV)}
    if own:
        import compressed_sparse_attention_index_gb300 as lib
        s["ws"] = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_EVICT, c["n_seq"], table.shape[1] * p),
                              dtype=torch.uint8, device=DEV)
    return s


def _prepare_verify(c, seed):
    g = _gen(seed)
    rows, V = _rows(c), c["vocab"]
    n, dt = sum(rows), {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[c["type"]]
    first = [0]
    for r in rows:
        first.append(first[-1] + r)
    greedy = c["mode"] == "greedy"
    target = torch.empty((n, V), dtype=dt, device=DEV)
    draft = torch.empty((n, V), dtype=dt, device=DEV) if c["draft_probs"] else None
    tokens = torch.randint(0, V, (n,), generator=g, device=DEV, dtype=torch.int32)
    for a in range(0, n, 64):
        b = min(n, a + 64)
        x = 2.5 * torch.randn((b - a, V), generator=g, device=DEV)
        target[a:b] = (x if greedy else torch.softmax(x, 1)).to(dt)
        if greedy:
            pick = _first_max(target[a:b])
        elif draft is None:
            pick = torch.multinomial(torch.softmax(1.5 * x, 1), 1, generator=g)[:, 0]
        else:
            draft[a:b] = torch.softmax(x + 0.7 * torch.randn((b - a, V), generator=g, device=DEV), 1).to(dt)
            pick = torch.multinomial(draft[a:b].float(), 1, generator=g)[:, 0]
        end = min(n, b + 1)
        tokens[a + 1:end] = pick[:end - a - 1].to(torch.int32)      # row t's proposal is the step's token t + 1
    if greedy:
        for i, a in enumerate(_agree(c)):                           # the first one that the target does not agree with
            if a + 1 < rows[i]:
                at = first[i] + a + 1
                tokens[at] = (tokens[at] + 1) % V
    s = {"op": "verify", "greedy": greedy, "n_seq": c["n_seq"], "n_rows": n, "vocab": V, "type": c["type"],
         "target": target, "draft": draft, "tokens": tokens, "first": _i32(first), "most": max(rows),
         "u": torch.rand(n, generator=g, device=DEV), "v": torch.rand(c["n_seq"], generator=g, device=DEV),
         "kept": torch.empty(c["n_seq"], dtype=torch.int32, device=DEV),
         "next": torch.empty(c["n_seq"], dtype=torch.int32, device=DEV)}
    if own:
        import compressed_sparse_attention_index_gb300 as lib
        s["ws"] = torch.empty(max(1, lib.csa2_workspace_size(lib.CSA2_OP_VERIFY, n, V)), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    f = {"weigh": (_plain_weigh, _own_weigh), "evict": (_plain_evict, _own_evict),
         "verify": (_plain_verify, _own_verify)}[state["op"]]
    return f[1](state) if own else f[0](state)


def _own_weigh(s):
    import compressed_sparse_attention_index_gb300 as lib
    lib.csa2_attn_weight(s["q"], s["pages"], s["n_pages"], s["page"], s["table"], s["table"].shape[1], s["first"],
                         s["n_seq"], s["sel"], 0 if s["sel"] is None else s["sel"].shape[1], s["n_vis"], s["lse"],
                         s["n_q"], s["decay"], s["prior"], s["weight"], None, s["ws"], s["ws"].numel())
    return s["weight"]


def _own_evict(s):
    import compressed_sparse_attention_index_gb300 as lib
    lib.csa2_evict(s["pages"], s["weight"], s["n_pages"], s["page"], s["table"], s["table"].shape[1], s["seq_len"],
                   s["keep"], s["n_seq"], s["recent"], s["dst_pages"], s["dst_weight"], s["n_dst"], s["dst_table"],
                   s["dst_table"].shape[1], s["new_len"], s["from"], s["from"].shape[1], s["ws"], s["ws"].numel())
    return {"pages": s["dst_pages"], "weight": s["dst_weight"], "len": s["new_len"], "from": s["from"]}


def _own_verify(s):
    import compressed_sparse_attention_index_gb300 as lib
    dtype = {"f32": lib.CSA2_PROB_F32, "bf16": lib.CSA2_PROB_BF16, "f16": lib.CSA2_PROB_F16}[s["type"]]
    lib.csa2_verify_drafts(lib.CSA2_VERIFY_GREEDY if s["greedy"] else lib.CSA2_VERIFY_SAMPLE, s["target"],
                           s["target"].shape[1], s["draft"], 0 if s["draft"] is None else s["draft"].shape[1], dtype,
                           s["vocab"], s["tokens"], s["first"], s["n_seq"], s["n_rows"], s["u"], s["v"], s["kept"],
                           s["next"], s["ws"], s["ws"].numel())
    return {"kept": s["kept"], "next": s["next"]}


def _slots(s, b, j, table="table"):
    """Slots of entries j of sequence b."""
    return s[table][b][j // s["page"]].long() * s["page"] + j % s["page"]


def _plain_weigh(s):
    pairs, flat, w = _e2m1_pairs(), s["pages"].view(-1, KV_BYTES), s["weight"]
    q, g = s["q"].to(torch.float32), s["queries"]
    if s["sel"] is None:
        for b, n in enumerate(s["lens"]):
            qb, lse, vis = q[b * g:b * g + g], s["lse"][b * g:b * g + g], s["n_vis"][b * g:b * g + g]
            step = max(1, min(n, (1 << 18) // g))
            for a in range(0, n, step):
                j = torch.arange(a, min(n, a + step), device=DEV)
                at = _slots(s, b, j)
                k = _kv_values(flat[at], pairs)
                x = torch.matmul(qb.view(-1, D), k.t()).view(g, H, -1) * SCALE
                p = torch.exp(x - lse[:, :, None]).sum(1)
                got = torch.where(j < vis[:, None], p, torch.zeros((), device=DEV)).sum(0)
                w[at] = s["decay"] * s["prior"][at] + got
        return w
    for b, n in enumerate(s["lens"]):
        at = _slots(s, b, torch.arange(n, device=DEV))
        got = torch.zeros(n, device=DEV)
        for i in range(b * g, b * g + g):
            ok = s["sel"][i] >= 0
            j = torch.where(ok, s["sel"][i], torch.zeros((), dtype=torch.int32, device=DEV)).long()
            k = _kv_values(flat[at[j]], pairs)
            p = torch.exp(torch.matmul(q[i], k.t()) * SCALE - s["lse"][i][:, None]).sum(0)
            got.index_add_(0, j, torch.where(ok, p, torch.zeros((), device=DEV)))
        w[at] = s["decay"] * s["prior"][at] + got
    return w


def _plain_evict(s):
    flat, dst = s["pages"].view(-1, KV_BYTES), s["dst_pages"].view(-1, KV_BYTES)
    for b, (n, k) in enumerate(zip(s["lens"], s["kept"])):
        last = min(s["recent"], k)
        at = _slots(s, b, torch.arange(n, device=DEV))
        w = s["weight"][at]
        order = torch.sort(w[:n - last], descending=True, stable=True).indices
        j = torch.cat([torch.sort(order[:k - last]).values, torch.arange(n - last, n, device=DEV)])
        to = _slots(s, b, torch.arange(k, device=DEV), "dst_table")
        dst[to] = flat[at[j]]
        s["dst_weight"][to] = w[j]
        s["from"][b, :k] = j.to(torch.int32)
        s["new_len"][b] = k
    return {"pages": s["dst_pages"], "weight": s["dst_weight"], "len": s["new_len"], "from": s["from"]}


def _first_max(x):
    """The lowest index of each row's largest value."""
    top = x == x.amax(1, keepdim=True)
    i = torch.arange(x.shape[1], device=x.device)
    return torch.where(top, i, torch.full((), x.shape[1], device=x.device)).amin(1)


def _plain_verify(s):
    first, V = s["first"].long(), s["vocab"]
    count = first[1:] - first[:-1]
    t = torch.arange(s["most"] - 1, device=DEV)
    row = (first[:-1, None] + t).clamp(max=s["n_rows"] - 1)
    drafted = t + 1 < count[:, None]
    tok = s["tokens"].long()[(row + 1).clamp(max=s["n_rows"] - 1)]
    if s["greedy"]:
        best = _first_max(s["target"])
        ok = best[row] == tok
    else:
        # products and running sums in 64 bits: on which side of a border a number falls decides a token
        p = s["target"][row, tok].double()
        q = s["draft"][row, tok].double() if s["draft"] is not None else torch.ones_like(p)
        ok = s["u"].double()[row] * q < p
    accepted = torch.cumprod((ok & drafted).long(), 1).sum(1)
    at = first[:-1] + accepted
    if s["greedy"]:
        return {"kept": (1 + accepted).to(torch.int32), "next": best[at].to(torch.int32)}
    p = s["target"][at].double()
    refused = accepted + 1 < count
    if s["draft"] is not None:
        r = torch.where(refused[:, None], (p - s["draft"][at].double()).clamp(min=0.0), p)
    else:
        x = s["tokens"].long()[(at + 1).clamp(max=s["n_rows"] - 1)]
        out = refused[:, None] & (torch.arange(V, device=DEV) == x[:, None])
        r = torch.where(out, torch.zeros((), dtype=torch.float64, device=DEV), p)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p)
    c = torch.cumsum(r, 1)
    past = c > s["v"].double()[:, None] * c[:, -1:]
    i = torch.arange(V, device=DEV)
    nxt = torch.where(past, i, torch.full((), V, device=DEV)).amin(1)
    last = torch.where(r > 0, i, torch.zeros((), dtype=torch.long, device=DEV)).amax(1)
    return {"kept": (1 + accepted).to(torch.int32), "next": torch.minimum(nxt, last).to(torch.int32)}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _f64_fp4(rec):
    """Latents of records from the bit fields of their codes and scales."""
    nib = torch.stack([rec[:, :256] & 15, rec[:, :256] >> 4], -1).view(-1, D).to(torch.int16)
    e, m = (nib >> 1) & 3, nib & 1
    mag = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0))
    b = rec[:, 256:].to(torch.int16)
    se, sm = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(se == 0, sm * 2.0 ** -9, (1.0 + sm / 8.0) * torch.exp2(se.double() - 7.0))
    return torch.where((nib & 8) != 0, -mag, mag) * sc.repeat_interleave(16, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        # sequence by sequence, draft by draft
        kept, nxt = [], []
        first = s["first"].tolist()
        tokens, u, v = s["tokens"].tolist(), s["u"].double().tolist(), s["v"].double().tolist()
        for b in range(case["n_seq"]):
            r, end = first[b], first[b + 1]
            if s["greedy"]:
                while True:
                    x = s["target"][r].double()
                    best = int(torch.nonzero(x == x.max())[0].item())
                    if r + 1 == end or tokens[r + 1] != best:
                        break
                    r += 1
                kept.append(r - first[b] + 1), nxt.append(best)
                continue
            res = None
            while r + 1 < end:
                x = tokens[r + 1]
                q = float(s["draft"][r, x].double()) if s["draft"] is not None else 1.0
                p = float(s["target"][r, x].double())
                if u[r] * q >= p:
                    res = s["target"][r].double()
                    if s["draft"] is not None:
                        res = torch.relu(res - s["draft"][r].double())
                    else:
                        res[x] = 0.0
                    break
                r += 1
            kept.append(r - first[b] + 1)
            if res is None or float(res.sum()) <= 0.0:
                res = s["target"][r].double()
            some = torch.nonzero(res > 0)[:, 0]
            run_sum = torch.cumsum(res[some], 0)
            i = int(torch.searchsorted(run_sum, run_sum[-1:] * v[b], right=True).item())
            nxt.append(int(some[min(i, some.numel() - 1)].item()))
        return {"kept": _i32(kept), "next": _i32(nxt)}
    flat = s["pages"].view(-1, KV_BYTES)
    if case["op"] == "evict":
        for b, (n, k) in enumerate(zip(s["lens"], s["kept"])):
            j = torch.arange(n, device=DEV)
            at = _slots(s, b, j)
            # later entries first in rank, then heavier, then earlier ones: one sort after the other
            key = torch.where(j >= n - min(s["recent"], k), torch.full((), math.inf, dtype=torch.float64, device=DEV),
                              s["weight"][at].double())
            stay = torch.zeros(n, dtype=torch.bool, device=DEV)
            if k > 0:
                border = torch.topk(key, k).values[-1]
                stay = key > border
                tie = torch.nonzero(key == border)[:, 0]
                stay[tie[:k - int(stay.sum())]] = True
            src = torch.nonzero(stay)[:, 0]
            to = _slots(s, b, torch.arange(k, device=DEV), "dst_table")
            s["dst_pages"].view(-1, KV_BYTES)[to] = flat[at[src]]
            s["dst_weight"][to] = s["weight"][at[src]]
            s["from"][b, :k] = src.to(torch.int32)
        return {"pages": s["dst_pages"], "weight": s["dst_weight"], "len": _i32(s["kept"]), "from": s["from"]}
    w = torch.zeros(flat.shape[0], dtype=torch.float64, device=DEV)
    g = s["queries"]
    for b, n in enumerate(s["lens"]):
        w[_slots(s, b, torch.arange(n, device=DEV))] += s["decay"] * s["prior"][_slots(s, b, torch.arange(n, device=DEV))].double()
        for i in range(b * g, (b + 1) * g):
            seen = int(s["n_vis"][i])
            chosen = torch.arange(seen, device=DEV) if s["sel"] is None else s["sel"][i][s["sel"][i] >= 0].long()
            for j in chosen.split(1 << 18):
                at = _slots(s, b, j)
                logit = _f64_fp4(flat[at]) @ s["q"][i].double().T * SCALE
                w.index_add_(0, at, torch.exp(logit - s["lse"][i].double()).sum(1))
    return w
