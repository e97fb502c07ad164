"""Operators of a paged CSA2 cache: what is measured, and their plain forms.

Four operators that a server needs around the sparse decode path when its main
cache is kept in pages (blocks of records with a block table per sequence):

* plan   csa2_page_plan: block tables, cache slots and the per-token
         descriptors of a step, from the sequences' lengths;
* norm   csa2_qk_norm_rope: the norm of every query head and of the latent, the
         rotation of their last 64 dims, and the cache write, in one pass
         (read back through csa2_cache_read);
* read   csa2_cache_read: records at given slots back to 512-wide latents;
* attn   csa2_paged_attn: 64-head attention over the paged latents (all visible
         ones, or a selection) and the 128-token window.

`own` False: elementary torch operations, in 32 bits (64 where 32 lose what
matters), rounded once at the end.  `own` True: the library's entry points.
"""
import math

import torch

own = False

H, D, ROPE, OFF, SWA = 64, 512, 64, 448, 128
KV_BYTES, SWA_BYTES = 288, 528
BASE, EPS, SCALE = 10000.0, 1e-6, 1.0 / math.sqrt(512.0)
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the step plan of 8 decoding sequences (one new token each)
        {"name": "plan_decode_8", "op": "plan", "n_seq": 8, "max_len": 1 << 20, "tokens": 8, "page": 64},
        # a mixed step: 1,000 sequences, most of them decoding, prompts up to 131,072 new tokens in all
        {"name": "plan_mixed_1000", "op": "plan", "n_seq": 1000, "max_len": 65536, "tokens": 131072, "page": 64},
        # the single token of one decoding sequence
        {"name": "norm_1", "op": "norm", "n": 1, "queries": True, "page": 64},
        # draft positions of a few sequences: an odd number of tokens
        {"name": "norm_33", "op": "norm", "n": 33, "queries": True, "page": 16},
        # the 8,192-token prompt of the prefill workload
        {"name": "norm_8192", "op": "norm", "n": 8192, "queries": True, "page": 64},
        # one query's selected entries read back
        {"name": "read_512", "op": "read", "kind": "kv", "n": 512, "slots": 65536},
        # a long prefix read back, an odd number of records
        {"name": "read_500001", "op": "read", "kind": "kv", "n": 500_001, "slots": 1 << 20},
        # one short sequence (the 4,096-entry workload): latency
        {"name": "attn_1x4096", "op": "attn", "n_seq": 1, "drafts": 1, "n": 4096, "sel": 0, "page": 64, "ragged": False},
        # five draft positions of 8 sequences over their selected 512 entries
        {"name": "attn_sel_40x512", "op": "attn", "n_seq": 8, "drafts": 5, "n": 65536, "sel": 512, "page": 64,
         "ragged": False},
        # a served batch of unequal lengths, pages that do not divide the kernels' tiles
        {"name": "attn_ragged_33", "op": "attn", "n_seq": 33, "drafts": 1, "n": 40_001, "sel": 0, "page": 48,
         "ragged": True},
        # the 32 x 65,536 decode workload
        {"name": "attn_32x65536", "op": "attn", "n_seq": 32, "drafts": 1, "n": 65536, "sel": 0, "page": 64,
         "ragged": False},
        # the 8 x 1,048,576 long-context workload, dense
        {"name": "attn_8x1M", "op": "attn", "n_seq": 8, "drafts": 1, "n": 1 << 20, "sel": 0, "page": 128,
         "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "norm", "read", "attn", "attn"])
    page = rng.choice([16, 32, 48, 64, 100, 128])
    if op == "plan":
        n_seq = _log(rng, 1, 4000)
        return {"op": op, "n_seq": n_seq, "max_len": _log(rng, 500, 65_000),
                "tokens": n_seq + _log(rng, 1, 120_000), "page": page}
    if op == "norm":
        return {"op": op, "n": _log(rng, 1, 8000), "queries": rng.random() < 0.8, "page": page}
    if op == "read":
        return {"op": op, "kind": rng.choice(["kv", "swa"]), "n": _log(rng, 1, 400_000),
                "slots": rng.choice([100_003, 1 << 18])}
    n_seq, drafts = _log(rng, 1, 48), rng.choice([1, 1, 2, 5])
    n = min(_log(rng, 1, 1 << 20), 2_000_000 // (n_seq * drafts))
    return {"op": op, "n_seq": n_seq, "drafts": drafts, "n": n, "sel": rng.choice([0, 0, 512, rng.randint(1, 512)]),
            "page": page, "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------ shapes that follow from a case
def _mix(i):
    """A fixed spread of i over [0, 1)."""
    return (i * 2654435761 + 40503) % (1 << 32) / float(1 << 32)


def _attn_lens(c):
    """Entries of every sequence; the first is always the longest."""
    n = c["n"]
    if not c["ragged"]:
        return [n] * c["n_seq"]
    return [n] + [max(c["drafts"], int(n * _mix(i))) for i in range(1, c["n_seq"])]


def _attn_queries(c):
    """(sequence, visible entries) of every query: draft t of G sees up to itself."""
    g = c["drafts"]
    return [(s, max(1, n - g + t + 1)) for s, n in enumerate(_attn_lens(c)) for t in range(g)]


def _plan_lens(c):
    """(length, new tokens) of every sequence; the new tokens add up to at most c["tokens"]."""
    out, left = [], c["tokens"] - c["n_seq"]
    for i in range(c["n_seq"]):
        new = 0 if i % 9 == 8 else 1
        if i % 7 == 3 or i == 0:
            more = min(left, int(c["tokens"] * _mix(i) / 8))
            new, left = new + more, left - more
        out.append((int(c["max_len"] * _mix(i + 77)), new))
    return out


def work(case):
    if case["op"] == "plan":
        p = case["page"]
        lens = _plan_lens(case)
        taken = sum(-(-(a + b) // p) - -(-a // p) for a, b in lens)
        return {"bytes": 8 * len(lens) + 4 * len(lens) + 8 * taken + 7 * 4 * case["tokens"], "flops": 0}
    if case["op"] == "norm":
        q = 2 * 2 * H * D if case["queries"] else 0
        return {"bytes": case["n"] * (q + 2 * 2 * D + KV_BYTES + SWA_BYTES + 2 * 2 * D), "flops": 0}
    if case["op"] == "read":
        rec = KV_BYTES if case["kind"] == "kv" else SWA_BYTES
        return {"bytes": case["n"] * (rec + 2 * D + 4), "flops": 0}
    pairs = records = 0
    for s, vis in _attn_queries(case):
        got = min(case["sel"], vis) if case["sel"] else vis
        win = min(SWA, vis)
        pairs += got + win
    lens = _attn_lens(case)
    records = sum(min(n, case["sel"] * case["drafts"]) if case["sel"] else n for n in lens)
    nq = case["n_seq"] * case["drafts"]
    return {"bytes": records * KV_BYTES + case["n_seq"] * SWA * SWA_BYTES + nq * (2 * 2 * H * D + 4 * H),
            "flops": 4.0 * H * D * pairs}


# ------------------------------------------------------------------ record formats, elementary
def _e2m1_pairs():
    """[256, 2]: the two FP4 values of a byte, low nibble first."""
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    val = mag + [-m for m in mag]
    return torch.tensor([[val[b & 15], val[b >> 4]] for b in range(256)], dtype=torch.float32, device=DEV)


def _e8m0(b):
    """2^(b - 127) of scale bytes."""
    return torch.exp2(b.to(torch.float32) - 127.0)


def _kv_values(rec, pairs):
    """[n, 288] record bytes -> [n, 512] fp32 latents."""
    v = pairs.index_select(0, rec[:, :256].reshape(-1).to(torch.int32)).view(-1, 32, 16)
    s = rec[:, 256:].contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    return (v * s[:, :, None]).view(-1, D)


def _swa_values(rec):
    """[n, 528] window record bytes -> [n, 512] fp32."""
    v = rec[:, :D].contiguous().view(torch.float8_e4m3fn).to(torch.float32).view(-1, 16, 32)
    return (v * _e8m0(rec[:, D:])[:, :, None]).view(-1, D)


def _e2m1_code(y):
    """Nearest FP4 code (ties to the even code), saturating; -0 keeps its sign."""
    a = y.abs()
    # borders between neighbouring magnitudes; the upper code takes a tie where it is even
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    tie_up = torch.tensor([False, True, False, True, False, True, False], device=y.device)
    edge = torch.where(tie_up, torch.nextafter(edge, torch.zeros_like(edge)), edge)
    return torch.bucketize(a, edge, out_int32=True) + 8 * torch.signbit(y).to(torch.int32)


def _pow2_scale(amax, lim):
    """Exponent of the smallest power of two >= amax / lim, within [-127, 127]; amax = 0 gives -127."""
    e = torch.ceil(torch.log2(amax.double() / lim))
    e = torch.where(torch.exp2(e - 1) * lim >= amax.double(), e - 1, e)
    e = torch.where(torch.exp2(e) * lim < amax.double(), e + 1, e)
    return e.clamp(-127, 127)


def _pack_kv(x):
    """bf16 [n, 512] -> record bytes [n, 288]."""
    g = x.to(torch.float32).view(-1, 32, 16)
    amax = g.abs().amax(2)
    s8 = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.to(torch.float32)
    code = torch.where(s[:, :, None] > 0, _e2m1_code(g / s[:, :, None]), torch.zeros((), dtype=torch.int32, device=x.device))
    code = code.view(-1, 256, 2)
    nib = (code[:, :, 0] | (code[:, :, 1] << 4)).to(torch.uint8)
    return torch.cat([nib, s8.view(torch.uint8)], 1)


def _pack_swa(x):
    """bf16 [n, 512] -> window record bytes [n, 528]."""
    g = x.to(torch.float32).view(-1, 16, 32)
    amax = g.abs().amax(2)
    e = torch.where(amax > 0, _pow2_scale(amax, 448.0), torch.full((), -127.0, dtype=torch.float64, device=x.device))
    v = (g.double() * torch.exp2(-e)[:, :, None]).to(torch.float32).clamp(-448.0, 448.0)
    v = torch.where(amax[:, :, None] > 0, v, torch.zeros((), device=x.device))
    return torch.cat([v.to(torch.float8_e4m3fn).view(torch.uint8).view(-1, D), (e + 127).to(torch.uint8)], 1)


def _angles(pos):
    """[n, 32] rotation angles of positions, in 64 bits."""
    i = torch.arange(ROPE // 2, dtype=torch.float64, device=pos.device)
    return pos.double()[:, None] * BASE ** (-2.0 * i / ROPE)


# ------------------------------------------------------------------ states
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _random_records(g, n, pack, width):
    out = torch.empty((n, width), dtype=torch.uint8, device=DEV)
    step = 1 << 18
    for a in range(0, n, step):
        b = min(n, a + step)
        out[a:b] = pack(torch.randn((b - a, D), generator=g, device=DEV).bfloat16())
    return out


def prepare(case, seed):
    return {"plan": _prepare_plan, "norm": _prepare_norm, "read": _prepare_read, "attn": _prepare_attn}[case["op"]](case, seed)


def _prepare_plan(c, seed):
    g = _gen(seed)
    p, lens = c["page"], _plan_lens(c)
    cols = max(-(-(a + b) // p) for a, b in lens) + 1
    taken = sum(-(-(a + b) // p) - -(-a // p) for a, b in lens)
    held = sum(-(-a // p) for a, _ in lens)
    n_pages = held + taken + 64
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    have = _i32([-(-a // p) for a, _ in lens])
    first = torch.cumsum(have, 0) - have
    col = torch.arange(cols, device=DEV, dtype=torch.int32)
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    table = torch.where(col < have[:, None], perm[at.long()], torch.full((), -1, dtype=torch.int32, device=DEV))
    m = c["tokens"]
    return {"op": "plan", "page": p, "n_pages": n_pages, "swa_cap": 192, "tokens": m,
            "seq_len": _i32([a for a, _ in lens]), "new_len": _i32([b for _, b in lens]),
            "free": perm[held:].contiguous(), "table": table.contiguous(),
            "desc": torch.empty((7, m), dtype=torch.int32, device=DEV),
            "first": torch.empty(len(lens) + 1, dtype=torch.int32, device=DEV),
            "totals": torch.empty(2, dtype=torch.int32, device=DEV)}


def _prepare_norm(c, seed):
    g = _gen(seed)
    n, p = c["n"], c["page"]
    n_pages = 2 * (-(-n // p)) + 8
    far = int(torch.randint(0, 1_000_000, (1,), generator=g, device=DEV).item())
    s = {"op": "norm", "n": n, "queries": c["queries"],
         # the query and latent rows of a projection's output, before their norms
         "latent": (3.0 * torch.randn((n, D), generator=g, device=DEV)).bfloat16(),
         "latent_gain": 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV),
         "pos": (far + torch.arange(n, device=DEV)).to(torch.int32),
         "slot": torch.randperm(n_pages * p, generator=g, device=DEV)[:n].to(torch.int32),
         "swa_slot": torch.randperm(n + 128, generator=g, device=DEV)[:n].to(torch.int32),
         "pages": torch.zeros((n_pages, p, KV_BYTES), dtype=torch.uint8, device=DEV),
         "swa": torch.zeros((1, n + 128, SWA_BYTES), dtype=torch.uint8, device=DEV),
         "latent_out": torch.empty((n, D), dtype=torch.bfloat16, device=DEV),
         "kv_back": torch.empty((n, D), dtype=torch.bfloat16, device=DEV),
         "swa_back": torch.empty((n, D), dtype=torch.bfloat16, device=DEV)}
    if c["queries"]:
        s["q"] = (2.0 * torch.randn((n, H, D), generator=g, device=DEV)).bfloat16()
        s["q_gain"] = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
        s["q_out"] = torch.empty((n, H, D), dtype=torch.bfloat16, device=DEV)
    return s


def _prepare_read(c, seed):
    g = _gen(seed)
    kv = c["kind"] == "kv"
    cache = _random_records(g, c["slots"], _pack_kv if kv else _pack_swa, KV_BYTES if kv else SWA_BYTES)
    return {"op": "read", "kv": kv, "cache": cache, "n": c["n"],
            "slots": torch.randint(0, c["slots"], (c["n"],), generator=g, device=DEV, dtype=torch.int32),
            "out": torch.empty((c["n"], D), dtype=torch.bfloat16, device=DEV)}


def _prepare_attn(c, seed):
    g = _gen(seed)
    p, lens, qs = c["page"], _attn_lens(c), _attn_queries(c)
    pages = [-(-n // p) for n in lens]
    n_pages, cols = sum(pages) + 3, max(pages)
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    have = _i32(pages)
    first = torch.cumsum(have, 0) - have
    col = torch.arange(cols, device=DEV, dtype=torch.int32)
    table = torch.where(col < have[:, None], perm[(first[:, None] + col).clamp(max=n_pages - 1).long()],
                        torch.full((), -1, dtype=torch.int32, device=DEV))
    nq = len(qs)
    vis = _i32([v for _, v in qs])
    cap = SWA + c["drafts"] - 1
    pos = vis - 1
    cnt = vis.clamp(max=SWA)
    s = {"op": "attn", "page": p, "n_pages": n_pages, "n_seq": c["n_seq"], "n_q": nq, "longest": max(lens),
         "pages": _random_records(g, n_pages * p, _pack_kv, KV_BYTES).view(n_pages, p, KV_BYTES),
         "table": table.contiguous(), "swa_cap": cap,
         "swa": _random_records(g, c["n_seq"] * cap, _pack_swa, SWA_BYTES).view(c["n_seq"], cap, SWA_BYTES),
         "q": torch.randn((nq, H, D), generator=g, device=DEV).bfloat16(),
         "q_seq": _i32([b for b, _ in qs]), "n_vis": vis, "pos": pos, "swa_cnt": cnt,
         "swa_first": (vis - cnt) % cap, "sel": None,
         "out": torch.empty((nq, H, D), dtype=torch.bfloat16, device=DEV),
         "lse": torch.empty((nq, H), dtype=torch.float32, device=DEV)}
    if c["sel"]:
        # distinct visible entries in ascending order, -1 behind them: one of each of `sel` equal parts of the row
        k = c["sel"]
        u = torch.rand((nq, k), generator=g, device=DEV, dtype=torch.float64)
        a = torch.arange(k, device=DEV, dtype=torch.float64)
        v = vis.double()[:, None]
        long_row = ((a + u) * v / k).floor()
        lo, hi = (a * v / k).ceil(), ((a + 1) * v / k).ceil() - 1
        long_row = torch.minimum(torch.maximum(long_row, lo), hi)
        short_row = torch.where(a < v, a, torch.full((), -1.0, dtype=torch.float64, device=DEV))
        s["sel"] = torch.where(v >= k, long_row, short_row).to(torch.int32).contiguous()
    if own:
        import compressed_sparse_attention_index_gb300 as lib
        s["ws"] = torch.empty(max(1, lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, nq, 0)), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    f = {"plan": (_plain_plan, _own_plan), "norm": (_plain_norm, _own_norm), "read": (_plain_read, _own_read),
         "attn": (_plain_attn, _own_attn)}[state["op"]]
    return f[1](state) if own else f[0](state)


def _own_plan(s):
    import compressed_sparse_attention_index_gb300 as lib
    lib.csa2_page_plan(s["seq_len"], s["new_len"], s["seq_len"].shape[0], s["page"], s["n_pages"], s["free"],
                       s["free"].shape[0], None, s["table"], s["table"].shape[1], s["swa_cap"], s["desc"], s["tokens"],
                       s["first"], s["totals"])
    return {"desc": s["desc"], "first": s["first"], "totals": s["totals"], "table": s["table"]}


def _own_norm(s):
    import compressed_sparse_attention_index_gb300 as lib
    n, q = s["n"], s["queries"]
    lib.csa2_qk_norm_rope(s["q"] if q else None, H * D, s["q_gain"] if q else None, s["q_out"] if q else None,
                          s["latent"], D, s["latent_gain"], s["latent_out"], s["pos"], s["slot"], s["swa_slot"], n,
                          EPS, s["pages"], s["pages"].shape[0] * s["pages"].shape[1], s["swa"], s["swa"].shape[1])
    lib.csa2_cache_read(lib.CSA2_KV_NVFP4, s["pages"], s["pages"].shape[0] * s["pages"].shape[1], s["slot"], n,
                        s["kv_back"], lib.CSA2_OUT_BF16)
    lib.csa2_cache_read(lib.CSA2_SWA_MXFP8, s["swa"], s["swa"].shape[1], s["swa_slot"], n, s["swa_back"],
                        lib.CSA2_OUT_BF16)
    out = {"latent": s["latent_out"], "kv": s["kv_back"], "window": s["swa_back"]}
    if q:
        out["q"] = s["q_out"]
    return out


def _own_read(s):
    import compressed_sparse_attention_index_gb300 as lib
    lib.csa2_cache_read(lib.CSA2_KV_NVFP4 if s["kv"] else lib.CSA2_SWA_MXFP8, s["cache"], s["cache"].shape[0],
                        s["slots"], s["n"], s["out"], lib.CSA2_OUT_BF16)
    return s["out"]


def _own_attn(s):
    import compressed_sparse_attention_index_gb300 as lib
    lib.csa2_paged_attn(s["q"], s["pages"], s["n_pages"], s["page"], s["table"], s["table"].shape[1], s["n_seq"],
                        s["sel"], 0 if s["sel"] is None else s["sel"].shape[1], s["swa"], s["swa_cap"], s["q_seq"],
                        s["n_vis"], s["pos"], s["swa_first"], s["swa_cnt"], s["n_q"], s["out"], lib.CSA2_OUT_BF16,
                        s["lse"], None, s["ws"], s["ws"].numel())
    return {"out": s["out"], "lse": s["lse"]}


def _plain_plan(s):
    p, cap, m = s["page"], s["swa_cap"], s["tokens"]
    ln, new, table = s["seq_len"].long(), s["new_len"].long(), s["table"]
    n_seq, cols = table.shape
    end = ln + new
    have, need = (ln + p - 1) // p, (end + p - 1) // p
    cu = torch.cumsum(new, 0)
    cp = torch.cumsum(need - have, 0)
    # the new pages, in sequence order, from the head of the free list
    j = torch.arange(s["free"].shape[0], device=DEV)
    b = torch.searchsorted(cp, j, right=True).clamp(max=n_seq - 1)
    col = have[b] + j - (cp[b] - (need - have)[b])
    at = torch.where(j < cp[-1], b * cols + col, torch.full((), n_seq * cols, device=DEV))
    flat = torch.cat([table.view(-1), table.new_zeros(1)])
    flat[at] = s["free"]
    table = flat[:-1].view(n_seq, cols)
    # the new tokens, in sequence order
    t = torch.arange(m, device=DEV)
    live = t < cu[-1]
    b = torch.searchsorted(cu, t, right=True).clamp(max=n_seq - 1)
    pos = torch.where(live, ln[b] + t - (cu[b] - new[b]), torch.zeros((), dtype=torch.long, device=DEV))
    page = table[b, pos // p].long()
    vis = pos + 1
    cnt = vis.clamp(max=min(SWA, cap))
    none = torch.full((), -1, dtype=torch.long, device=DEV)
    zero = torch.zeros((), dtype=torch.long, device=DEV)
    rows = [torch.where(live, b, zero), torch.where(live, vis, zero), pos, torch.where(live, (vis - cnt) % cap, zero),
            torch.where(live, cnt, zero), torch.where(live, page * p + pos % p, none),
            torch.where(live & (pos + cap >= end[b]), b * cap + pos % cap, none)]
    return {"desc": torch.stack(rows).to(torch.int32), "first": torch.cat([cu.new_zeros(1), cu]).to(torch.int32),
            "totals": torch.stack([cu[-1], cp[-1]]).to(torch.int32), "table": table}


def _norm_rotated(x, gain, pos, f):
    """[n, h, 512] rows -> normed, scaled and rotated forward by pos, computed in f."""
    x = x.to(f)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(f)
    th = _angles(pos)
    c, sn = torch.cos(th).to(f)[:, None], torch.sin(th).to(f)[:, None]
    a, b = y[..., OFF::2], y[..., OFF + 1::2]
    r = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
    return torch.cat([y[..., :OFF], r], -1)


def _round_bf16(x):
    """64-bit values to bf16, rounded once (the conversion through 32 bits would round twice)."""
    m, e = torch.frexp(x)
    r = torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, 8))), e - 8)
    return r.to(torch.bfloat16)


def _plain_norm(s):
    # latents in 64 bits: their records hang on which side of a rounding border a value falls
    lat = _round_bf16(_norm_rotated(s["latent"][:, None], s["latent_gain"], s["pos"], torch.float64)[:, 0])
    kv, win = _pack_kv(lat), _pack_swa(lat)
    s["pages"].view(-1, KV_BYTES)[s["slot"].long()] = kv
    s["swa"].view(-1, SWA_BYTES)[s["swa_slot"].long()] = win
    out = {"latent": lat,
           "kv": _kv_values(s["pages"].view(-1, KV_BYTES)[s["slot"].long()], _e2m1_pairs()).bfloat16(),
           "window": _swa_values(s["swa"].view(-1, SWA_BYTES)[s["swa_slot"].long()]).bfloat16()}
    if s["queries"]:
        out["q"] = _norm_rotated(s["q"], s["q_gain"], s["pos"], torch.float32).bfloat16()
    return out


def _plain_read(s):
    rec = s["cache"].index_select(0, s["slots"])
    return (_kv_values(rec, _e2m1_pairs()) if s["kv"] else _swa_values(rec)).bfloat16()


def _plain_attn(s):
    nq, p, q = s["n_q"], s["page"], s["q"].to(torch.float32)
    seq = s["q_seq"].long()
    if s["sel"] is None:
        idx = torch.arange(s["longest"], device=DEV)[None].expand(nq, -1)
        ok = idx < s["n_vis"][:, None]
    else:
        idx, ok = s["sel"].long(), s["sel"] >= 0
    idx = torch.where(ok, idx, torch.zeros((), dtype=torch.long, device=DEV))
    page = torch.gather(s["table"][seq], 1, idx // p).long()
    slot = (page * p + idx % p).view(-1)
    k = _kv_values(s["pages"].view(-1, KV_BYTES)[slot], _e2m1_pairs()).view(nq, -1, D)
    t = torch.arange(SWA, device=DEV)
    wok = t < s["swa_cnt"][:, None]
    ring = seq[:, None] * s["swa_cap"] + (s["swa_first"][:, None] + t) % s["swa_cap"]
    w = _swa_values(s["swa"].view(-1, SWA_BYTES)[ring.view(-1)]).view(nq, -1, D)
    inf = torch.full((), -math.inf, device=DEV)
    lk = torch.where(ok[:, None], torch.bmm(q, k.transpose(1, 2)) * SCALE, inf)
    lw = torch.where(wok[:, None], torch.bmm(q, w.transpose(1, 2)) * SCALE, inf)
    m = torch.maximum(lk.amax(-1, keepdim=True), lw.amax(-1, keepdim=True))
    lk, lw = torch.exp(lk - m), torch.exp(lw - m)
    total = lk.sum(-1, keepdim=True) + lw.sum(-1, keepdim=True)
    o = (torch.bmm(lk, k) + torch.bmm(lw, w)) / total
    th = _angles(s["pos"])
    c, sn = torch.cos(th).float()[:, None], torch.sin(th).float()[:, None]
    a, b = o[..., OFF::2], o[..., OFF + 1::2]
    r = torch.stack([a * c + b * sn, b * c - a * sn], -1).flatten(-2)
    return {"out": torch.cat([o[..., :OFF], r], -1).bfloat16(), "lse": (m + torch.log(total))[..., 0]}


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


def _f64_fp8(rec):
    b = rec[:, :D].to(torch.int16)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0))
    sc = torch.exp2(rec[:, D:].double() - 127.0)
    return torch.where((b & 128) != 0, -mag, mag) * sc.repeat_interleave(32, 1)


def _f64_grid(x, points):
    """The nearest of ascending non-negative `points` to |x|, ties to the one of even number, with x's sign."""
    a = x.abs().clamp(max=float(points[-1]))
    hi = torch.searchsorted(points, a.contiguous()).clamp(min=1, max=points.numel() - 1)
    lo = hi - 1
    dl, dh = a - points[lo], points[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(points[pick], x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "read":
        rec = s["cache"][s["slots"].long()]
        return _f64_fp4(rec) if s["kv"] else _f64_fp8(rec)
    if case["op"] == "norm":
        def rows(x, gain):
            x = x.double()
            y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS) * gain.double()
            z = torch.view_as_complex(y[..., OFF:].reshape(*y.shape[:-1], ROPE // 2, 2).contiguous())
            f = torch.tensor([BASE ** (-i / 32.0) for i in range(32)], dtype=torch.float64, device=DEV)
            th = torch.outer(s["pos"].double(), f).view(x.shape[0], *([1] * (x.dim() - 2)), 32)
            y[..., OFF:] = torch.view_as_real(z * torch.polar(torch.ones_like(th), th)).flatten(-2)
            return y
        lat = rows(s["latent"], s["latent_gain"])
        e = torch.floor(torch.log2(lat.abs().clamp(min=1e-300))) - 7
        b = torch.round(lat * torch.exp2(-e)) * torch.exp2(e)      # the bf16 that the records are made of
        e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)]
                            + [(1 + m / 8) * 2.0 ** (k - 7) for k in range(1, 16) for m in range(8)][:-1],
                            dtype=torch.float64, device=DEV)
        g = b.view(-1, 32, 16)
        sc = _f64_grid(g.abs().amax(2) / 6.0, e4m3)[..., None]
        kv = torch.where(sc > 0, _f64_grid(g / sc.clamp(min=1e-300), e2m1) * sc, torch.zeros_like(g)).view(-1, D)
        g = b.view(-1, 16, 32)
        top = g.abs().amax(2)[..., None]
        # the smallest power of two p with 448 p >= top
        p = torch.exp2(torch.arange(-60, 61, device=DEV, dtype=torch.float64))
        p = p[torch.searchsorted(p * 448.0, top.contiguous())]
        out = {"latent": lat, "kv": kv, "window": (_f64_grid(g / p, e4m3) * p).view(-1, D)}
        if case["queries"]:
            out["q"] = rows(s["q"], s["q_gain"])
        return out
    outs, lses = [], []
    flat, swa = s["pages"].view(-1, KV_BYTES), s["swa"]
    f = torch.tensor([BASE ** (-i / 32.0) for i in range(32)], dtype=torch.float64, device=DEV)
    for i, (b, vis) in enumerate(_attn_queries(case)):
        j = torch.arange(vis, device=DEV) if s["sel"] is None else s["sel"][i][s["sel"][i] >= 0].long()
        at = s["table"][b].long()[j // s["page"]] * s["page"] + j % s["page"]
        ring = (int(vis - min(vis, SWA)) + torch.arange(min(vis, SWA), device=DEV)) % s["swa_cap"]
        k = torch.cat([_f64_fp4(flat[at]), _f64_fp8(swa[b][ring])])
        logit = (k @ s["q"][i].double().T) * SCALE
        lse = torch.logsumexp(logit, 0)
        o = torch.exp(logit - lse).T @ k
        z = torch.view_as_complex(o[:, OFF:].reshape(H, 32, 2).contiguous())
        th = (vis - 1) * f
        o[:, OFF:] = torch.view_as_real(z * torch.polar(torch.ones_like(th), -th)).flatten(-2)
        outs.append(o)
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
