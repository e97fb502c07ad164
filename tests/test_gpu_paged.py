"""GPU parity of the paged-cache operators against their 64-bit restatements
(tests/paged_reference.py), through the C ABI: integers and cache bytes
exactly, attention within the library's bound (2e-3 row-normalised in fp32, one
bf16 rounding more in bf16)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gen import inputs as G  # noqa: E402
from tests import paged_reference as R  # noqa: E402
from tests.parity import ATTN_TOL_BF16, ATTN_TOL_F32, row_norm_err  # noqa: E402

BOUNDS = 4


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


def _i32(x):
    return torch.from_numpy(np.array(x, np.int32)).cuda()


def _bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


# ------------------------------------------------------------------ plan
def _run_plan(lib, seq_len, new_len, page, n_pages, free, head, table, cap, max_tokens):
    table = np.array(table, np.int32)
    n_seq, stride = table.shape
    t = _i32(table)
    desc = torch.full((7, max(max_tokens, 1)), -77, dtype=torch.int32, device="cuda")
    first = torch.full((n_seq + 1,), -77, dtype=torch.int32, device="cuda")
    totals = torch.full((2,), -77, dtype=torch.int32, device="cuda")
    lib.csa2_page_plan(_i32(seq_len), _i32(new_len), n_seq, page, n_pages, _i32(free), len(free),
                       None if head is None else _i32([head]), t, stride, cap, desc, max_tokens, first, totals)
    st = lib.csa2_get_device_status()
    want = R.plan(seq_len, new_len, page, n_pages, free, head or 0, table, cap, max_tokens)
    if max_tokens:
        assert np.array_equal(desc.cpu().numpy(), want[0])
    assert np.array_equal(first.cpu().numpy(), want[1])
    assert np.array_equal(totals.cpu().numpy(), want[2])
    assert np.array_equal(t.cpu().numpy(), want[3])
    assert st == (0 if want[4] else BOUNDS)
    return want


@pytest.mark.parametrize("n_seq,page,max_len,max_new,cap,seed", [
    (1, 64, 0, 1, 128, 0), (1, 1, 40, 9, 128, 1), (5, 48, 500, 3, 130, 2), (130, 16, 300, 2, 192, 3),
    (700, 100, 2000, 40, 128, 4), (3000, 64, 900, 1, 1, 5), (9, 64, 100, 5000, 128, 6), (40, 7, 50, 60, 0, 7)])
def test_plan(lib, n_seq, page, max_len, max_new, cap, seed):
    r = np.random.default_rng(seed)
    ln, new = r.integers(0, max_len + 1, n_seq), r.integers(0, max_new + 1, n_seq)
    cols = -(-(max_len + max_new) // page) + 1
    n_pages = n_seq * cols + 5
    ids = r.permutation(n_pages).astype(np.int64)
    table = np.full((n_seq, cols), -1, np.int64)
    k = 0
    for b in range(n_seq):
        have = -(-int(ln[b]) // page)
        table[b, :have] = ids[k:k + have]
        k += have
    tokens = int(new.sum())
    want = _run_plan(lib, ln, new, page, n_pages, ids[k:], None, table, cap, tokens + 13)
    assert want[4]                                       # nothing out of range here
    _run_plan(lib, ln, new, page, n_pages, ids, k, table, cap, tokens)


def test_plan_of_no_sequences_and_no_tokens(lib):
    desc = torch.full((7, 40), -77, dtype=torch.int32, device="cuda")
    first, totals = torch.full((1,), -77, dtype=torch.int32, device="cuda"), torch.full((2,), -77, dtype=torch.int32, device="cuda")
    lib.csa2_page_plan(None, None, 0, 64, 10, None, 0, None, None, 1, 128, desc, 40, first, totals)
    assert first.tolist() == [0] and totals.tolist() == [0, 0] and lib.csa2_get_device_status() == 0
    assert np.array_equal(desc.cpu().numpy(), np.repeat([[0], [0], [0], [0], [0], [-1], [-1]], 40, 1))
    _run_plan(lib, [5, 70], [0, 0], 64, 10, [], None, [[1, 2], [3, 4]], 128, 0)


def test_plan_out_of_range(lib):
    table = np.array([[3, -1], [4, 5], [-1, 2], [99, 1], [6, -1]])
    # a negative length, a row that is too short, a column that names no page (twice), a free list that ends
    _run_plan(lib, [-1, 60, 20, 70, 64], [3, 100, 2, 1, 2], 64, 100, [7], None, table, 128, 32)
    _run_plan(lib, [10, 60, 20, 5, 64], [3, 2, 2, -4, 2], 64, 50, [7, 8], None, table, 128, 32)
    _run_plan(lib, [64, 64], [1, 1], 64, 50, [500, -3], None, [[1, 2], [3, 4]], 128, 4)       # free ids that name no page
    _run_plan(lib, [64, 64], [1, 1], 64, 50, [5, 6], -1, [[1, 2], [3, 4]], 128, 4)            # a head before the list
    _run_plan(lib, [0, 0, 0], [5, 5, 5], 4, 50, [5, 6, 7, 8, 9, 10], None, np.full((3, 2), -1), 128, 8)   # tokens beyond the descriptors
    _run_plan(lib, [2**31 - 1, 5], [1, 1], 1 << 20, 2000, [5, 6], None, np.zeros((2, 3000), np.int64), 128, 4)


def test_plan_largest_number_of_sequences(lib):
    r = np.random.default_rng(9)
    n = 16384
    ln, new = r.integers(0, 64, n), r.integers(0, 3, n)
    _run_plan(lib, ln, new, 32, 40000, r.permutation(40000), None, np.zeros((n, 3), np.int64) + 7, 128, int(new.sum()))


# ------------------------------------------------------------------ norm, rotation, cache write
def _norm_case(n, seed, scale=2.0):
    q = (G.normal_block_bf16(seed, G.S_Q, 1, 0, n * 64, 512)).reshape(n, 64, 512)
    lat = G.normal_block_bf16(seed, G.S_LATENT, 1, 0, n, 512)
    r = np.random.default_rng(seed)
    gain = (1 + 0.2 * r.normal(size=(2, 512))).astype(np.float32)
    pos = r.integers(0, 1 << 20, n)
    return q, lat, gain, pos


def _check_q(out_bits, q, gain, pos, eps):
    ref = R.norm_rope(R.bf16_values(q), gain, np.asarray(pos)[:, None], eps)
    # one bf16 rounding, and fp32: 16 terms and 5 joins of the sum (2^-20), the quotient and
    # products (2^-22), cos and sin (2^-22) of a pair's |a| + |b|
    room = np.abs(ref)
    room[..., 448::2] += np.abs(ref[..., 449::2])
    room[..., 449::2] += np.abs(ref[..., 448::2])
    assert np.all(np.abs(R.bf16_values(out_bits) - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-18 * room + 2.0**-133)


@pytest.mark.parametrize("n,gains,strided", [(1, True, False), (1, False, True), (7, True, True), (33, True, False),
                                             (160, False, False), (310, True, False), (650, True, True)])
def test_norm_rope_and_write(lib, oracle_lib, n, gains, strided):
    q, lat, gain, pos = _norm_case(n, 400 + n)
    eps = 1e-6
    pad = 24 if strided else 0
    qs, ls = 32768 + pad, 512 + pad
    qd = torch.full((n, qs), float("nan"), dtype=torch.bfloat16, device="cuda")
    qd[:, :32768] = _bf16(q.reshape(n, -1))
    ld = torch.full((n, ls), float("nan"), dtype=torch.bfloat16, device="cuda")
    ld[:, :512] = _bf16(lat)
    r = np.random.default_rng(n)
    slots, wslots = r.permutation(n + 9)[:n], r.permutation(n + 5)[:n]
    slots[n // 2] = -1                                     # one row is not written
    kv = torch.full((n + 9, 288), 0xAB, dtype=torch.uint8, device="cuda")
    swa = torch.full((n + 5, 528), 0xCD, dtype=torch.uint8, device="cuda")
    q_out = torch.empty((n, 64, 512), dtype=torch.bfloat16, device="cuda")
    l_out = torch.empty((n, 512), dtype=torch.bfloat16, device="cuda")
    g = torch.from_numpy(gain).cuda()
    lib.csa2_qk_norm_rope(qd, qs, g[0].contiguous() if gains else None, q_out, ld, ls, g[1].contiguous() if gains else None,
                          l_out, _i32(pos), _i32(slots), _i32(wslots), n, eps, kv, n + 9, swa, n + 5)
    assert lib.csa2_get_device_status() == 0
    _check_q(_bits(q_out), q, gain[0] if gains else None, pos, eps)
    want = R.round_bf16_bits(R.norm_rope(R.bf16_values(lat), gain[1] if gains else None, pos, eps))
    assert np.array_equal(_bits(l_out), want)
    rec, win = np.full((n + 9, 288), 0xAB, np.uint8), np.full((n + 5, 528), 0xCD, np.uint8)
    rec[slots[slots >= 0]] = oracle_lib.pack_kv(want)[slots >= 0]
    win[wslots] = oracle_lib.pack_swa(want)
    assert np.array_equal(kv.cpu().numpy(), rec) and np.array_equal(swa.cpu().numpy(), win)


def test_norm_latents_at_the_edges_of_their_range(lib, oracle_lib):
    """Zero rows, subnormal and huge rows, gains that under- or overflow, far positions: still the exact value's rounding."""
    from tests.test_gpu_pack_topk import _edge_rows
    x = _edge_rows(512)
    n = x.shape[0]
    r = np.random.default_rng(3)
    gain = np.where(r.random(512) < 0.1, 0.0, r.normal(size=512) * 10.0 ** r.integers(-30, 6, 512)).astype(np.float32)
    pos = np.array([0, 1, 2**31 - 1, 2**20, 3, 77, 10**6, 5, 6, 2**30 + 1, 8, 9][:n])
    for eps in (1e-6, 1e-12):
        out = torch.empty((n, 512), dtype=torch.bfloat16, device="cuda")
        kv = torch.zeros((n, 288), dtype=torch.uint8, device="cuda")
        lib.csa2_qk_norm_rope(None, 0, None, None, _bf16(x), 512, torch.from_numpy(gain).cuda(), out, _i32(pos),
                              _i32(np.arange(n)), None, n, eps, kv, n, None, 0)
        ref = R.norm_rope(R.bf16_values(x), gain, pos, eps)
        got, want = _bits(out), R.round_bf16_bits(ref)
        # angles beyond 2^28 are known to 2^-24 only in fp64 (pos * freq is rounded to 53 bits): those rows
        # are held to that, the others to equality
        far = pos >= 2**28
        assert np.array_equal(got[~far] & np.where(want[~far] & 0x7FFF, 0xFFFF, 0x7FFF), want[~far] & np.where(want[~far] & 0x7FFF, 0xFFFF, 0x7FFF))
        room = np.abs(ref)
        room[:, 448::2] += np.abs(ref[:, 449::2])
        room[:, 449::2] += np.abs(ref[:, 448::2])
        assert np.all(np.abs(R.bf16_values(got)[far] - ref[far]) <= 2.0**-8 * np.abs(ref[far]) + 2.0**-20 * room[far] + 2.0**-133)
        assert np.array_equal(kv.cpu().numpy(), oracle_lib.pack_kv(got))


def test_norm_in_place_parts_alone_and_out_of_range_slots(lib, oracle_lib):
    n = 20
    q, lat, gain, pos = _norm_case(n, 55)
    qd, ld = _bf16(q), _bf16(lat)
    g = torch.from_numpy(gain).cuda()
    # queries alone, in place
    lib.csa2_qk_norm_rope(qd, 32768, g[0].contiguous(), qd, None, 0, None, None, _i32(pos), None, None, n, 1e-5, None, 0, None, 0)
    _check_q(_bits(qd), q, gain[0], pos, 1e-5)
    # latents alone, in place, some slots out of range: skipped and reported
    slots = np.arange(n)
    slots[[3, 9]] = [n, 2**31 - 1]
    kv = torch.full((n, 288), 0xAB, dtype=torch.uint8, device="cuda")
    lib.csa2_qk_norm_rope(None, 0, None, None, ld, 512, None, ld, _i32(pos), _i32(slots), None, n, 1e-5, kv, n, None, 0)
    assert lib.csa2_get_device_status() == BOUNDS
    want = R.round_bf16_bits(R.norm_rope(R.bf16_values(lat), None, pos, 1e-5))
    rec = oracle_lib.pack_kv(want)
    rec[[3, 9]] = 0xAB
    assert np.array_equal(_bits(ld), want) and np.array_equal(kv.cpu().numpy(), rec)
    # window records alone
    swa = torch.full((n, 528), 0xCD, dtype=torch.uint8, device="cuda")
    lib.csa2_qk_norm_rope(None, 0, None, None, _bf16(lat), 512, None, None, _i32(pos), None, _i32(np.arange(n)[::-1]), n, 1e-5,
                          None, 0, swa, n)
    assert np.array_equal(swa.cpu().numpy(), oracle_lib.pack_swa(want)[::-1]) and lib.csa2_get_device_status() == 0


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("n", [1, 5, 1000, 40_003])
@pytest.mark.parametrize("kind", ["kv", "swa"])
@pytest.mark.parametrize("f32", [False, True])
def test_read(lib, oracle_lib, n, kind, f32):
    x = G.normal_block_bf16(91, G.S_MISC, 2, 0, 300, 512)
    rec = oracle_lib.pack_kv(x) if kind == "kv" else oracle_lib.pack_swa(x)
    val = R.kv_values(rec) if kind == "kv" else R.swa_values(rec)
    r = np.random.default_rng(n)
    slots = r.integers(0, 300, n)
    if n > 1:
        slots[::7] = -1 - slots[::7]                      # none: zeros
        slots[3] = 300                                    # behind the cache: zeros, reported
    out = torch.full((n + 2, 512), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lib.csa2_cache_read(lib.CSA2_KV_NVFP4 if kind == "kv" else lib.CSA2_SWA_MXFP8, torch.from_numpy(rec).cuda(), 300, _i32(slots),
                        n, out, lib.CSA2_OUT_F32 if f32 else lib.CSA2_OUT_BF16)
    assert lib.csa2_get_device_status() == (BOUNDS if n > 1 else 0)
    want = np.where(((slots >= 0) & (slots < 300))[:, None], val[np.clip(slots, 0, 299)], 0.0)
    got = out.float().cpu().numpy()
    assert np.array_equal(got[:n], want) and np.all(got[n:] == 7.0)


# ------------------------------------------------------------------ attention
class Case:
    """A paged cache of sequences of the given lengths, with NaN scales in every record that no sequence holds."""

    def __init__(self, oracle_lib, lens, page, swa_cap=128, seed=0, latent_scale=1.0, swa_scale=1.0):
        r = np.random.default_rng(seed)
        self.lens, self.page, self.swa_cap = list(lens), page, swa_cap
        cols = max(1, max(-(-n // page) for n in lens)) + 1
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + 3
        ids = r.permutation(self.n_pages)
        self.table = np.full((len(lens), cols), -1, np.int64)
        self.pages = np.full((self.n_pages, page, 288), 0xFF, np.uint8)
        k = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = ids[k:k + need[b]]
            k += need[b]
            x = R.bf16_values(G.normal_block_bf16(seed + 7, G.S_LATENT, b, 0, max(n, 1), 512)) * np.float32(latent_scale)
            rec = oracle_lib.pack_kv(R.round_bf16_bits(x))
            for j in range(n):
                self.pages[self.table[b, j // page], j % page] = rec[j]
        x = R.bf16_values(G.normal_block_bf16(seed + 8, G.S_SWA, 0, 0, len(lens) * max(swa_cap, 1), 512)) * np.float32(swa_scale)
        self.swa = oracle_lib.pack_swa(R.round_bf16_bits(x)).reshape(len(lens), max(swa_cap, 1), 528)

    def run(self, lib, queries, q_scale=1.0, sel=None, f32=True, lse=True, fill=0xA5, seed=1, table=None, stream=None):
        """queries: (sequence, n_vis, pos, swa_first, swa_cnt)."""
        nq = len(queries)
        a = np.array(queries, np.int64).reshape(nq, 5)
        x = R.bf16_values(G.normal_block_bf16(seed, G.S_Q, 3, 0, nq * 64, 512)) * np.float32(q_scale)
        self.q = R.round_bf16_bits(x).reshape(nq, 64, 512)
        wsb = lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, nq, 0)
        ws = torch.full((wsb,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((nq + 1, 64, 512), 5.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        le = torch.full((nq + 1, 64), 5.0, dtype=torch.float32, device="cuda") if lse else None
        table = self.table if table is None else table
        lib.csa2_paged_attn(_bf16(self.q), torch.from_numpy(self.pages).cuda(), self.n_pages, self.page, _i32(table),
                            table.shape[1], len(self.lens), None if sel is None else _i32(sel),
                            0 if sel is None else sel.shape[1], torch.from_numpy(self.swa).cuda() if self.swa_cap else None,
                            self.swa_cap, _i32(a[:, 0]), _i32(a[:, 1]), _i32(a[:, 2]), _i32(a[:, 3]), _i32(a[:, 4]), nq, out,
                            lib.CSA2_OUT_F32 if f32 else lib.CSA2_OUT_BF16, le, None, ws, wsb)
        torch.cuda.synchronize()
        assert bool((out[nq:] == 5.0).all()) and (le is None or bool((le[nq:] == 5.0).all()))      # rows behind: left as they were
        return out[:nq].float().cpu().numpy(), None if le is None else le[:nq].cpu().numpy()

    def want(self, queries, i, sel=None, table=None):
        b, vis, pos, first, cnt = queries[i]
        table = self.table if table is None else table
        idx = range(vis) if sel is None else [j for j in sel[i] if 0 <= j < vis]
        k = R.kv_values(R.paged_rows(self.pages, table[b], self.page, idx))
        if cnt:
            ring = (first + np.arange(cnt)) % self.swa_cap
            k = np.concatenate([k, R.swa_values(self.swa[b][ring])])
        o, lse = R.attention(R.bf16_values(self.q[i]), k, pos)
        # fp32 accumulation of 512 products: 512 half steps of the sum of their magnitudes
        room = 2.0**-15 * 512**-0.5 * (np.abs(R.bf16_values(self.q[i]).astype(np.float64)) @ np.abs(k).T).max() if len(k) else 0.0
        return o, lse, room + 1e-6

    def check(self, lib, queries, got=None, sel=None, f32=True, table=None, **kw):
        out, lse = got if got is not None else self.run(lib, queries, sel=sel, f32=f32, table=table, **kw)
        for i in range(len(queries)):
            o, le, room = self.want(queries, i, sel, table)
            assert row_norm_err(out[i], o) <= (ATTN_TOL_F32 if f32 else ATTN_TOL_BF16), i
            if lse is not None:
                if np.isinf(le).all():
                    assert np.array_equal(lse[i], le.astype(np.float32))
                else:
                    assert np.abs(lse[i] - le).max() <= room + 2.0**-23 * np.abs(le).max(), (i, np.abs(lse[i] - le).max(), room)
        return out, lse


def _decode_queries(lens, cap=128):
    q = []
    for b, n in enumerate(lens):
        cnt = min(128, cap, n)
        q.append((b, n, max(n - 1, 0), (n - cnt) % cap if cap else 0, cnt))
    return q


@pytest.mark.parametrize("lens,page", [([1], 64), ([128], 128), ([127, 129, 1, 2], 64), ([640, 300], 48), ([257], 1),
                                       ([500, 0, 33], 200), ([5000], 64), ([2000, 1, 700, 1300, 4000], 129)])
@pytest.mark.parametrize("f32", [True, False])
def test_attn_dense(lib, oracle_lib, lens, page, f32):
    c = Case(oracle_lib, lens, page, seed=len(lens) + page)
    c.check(lib, _decode_queries(lens), f32=f32)
    assert lib.csa2_get_device_status() == 0


def test_attn_drafts_without_window_and_empty_rows(lib, oracle_lib):
    c = Case(oracle_lib, [900, 260], 64, swa_cap=140, seed=5)
    # several tokens of a sequence, each with its own length; no window; rows with nothing at all; a wrapping window
    q = [(0, 896 + t, 895 + t, 0, 0) for t in range(5)] + [(1, 0, 3, 0, 0), (1, 0, 70_001, 130, 128), (0, 900, 2**20, 139, 100),
                                                         (1, 256, 9, 0, 1), (1, 0, 0, 0, 0)]
    out, lse = c.check(lib, q)
    assert np.all(out[5] == 0) and np.all(out[9] == 0) and np.all(np.isneginf(lse[5]))
    assert lib.csa2_get_device_status() == 0
    d = Case(oracle_lib, [300], 64, swa_cap=0, seed=6)
    d.check(lib, [(0, 300, 299, 0, 0), (0, 17, 16, 0, 0)])
    # many rows with nothing beside one that has
    out, lse = c.check(lib, [(0, 0, 0, 0, 0)] * 400 + [(0, 700, 699, 0, 128)])
    assert np.all(out[:400] == 0)


@pytest.mark.parametrize("k", [1, 129, 512])
def test_attn_selection(lib, oracle_lib, k):
    c = Case(oracle_lib, [3000, 150], 48, seed=20 + k)
    r = np.random.default_rng(k)
    q = [(0, 3000, 2999, 5, 128), (0, 2500, 2499, 0, 0), (1, 150, 149, 22, 128), (1, 100, 99, 0, 100), (0, 0, 0, 0, 30)]
    sel = np.full((len(q), k), -1, np.int64)
    for i, (b, vis, *_ ) in enumerate(q):
        m = min(k, vis)
        sel[i, :m] = np.sort(r.permutation(vis)[:m])
    sel[0, ::3] = -1                                       # holes
    if k == 512:
        sel[1, 128:256] = -1                               # a whole tile of holes
        sel[2] = -1                                        # nothing selected: the window alone
    c.check(lib, q, sel=sel)
    assert lib.csa2_get_device_status() == 0
    # the same answer as csa2_sparse_attn over the contiguous cache
    flat = torch.from_numpy(np.stack([R.paged_rows(c.pages, c.table[0], 48, range(3000))])).cuda()
    sa = torch.empty((2, 64, 512), dtype=torch.float32, device="cuda")
    wsb = lib.csa2_workspace_size(lib.CSA2_OP_SPARSE_ATTN, 2, k + 128)
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device="cuda")
    a = np.array(q[:2])
    lib.csa2_sparse_attn(_bf16(c.q[:2]), flat, 3000, 1, _i32(sel[:2]), k, torch.from_numpy(c.swa[:1]).cuda(), 128, _i32(a[:, 0]), _i32(a[:, 2]),
                         _i32(a[:, 3]), _i32(a[:, 4]), 2, sa, lib.CSA2_OUT_F32, None, ws, wsb)
    out, _ = c.run(lib, q, sel=sel)
    assert row_norm_err(out[:2], sa.cpu().numpy()) <= 2 * ATTN_TOL_F32


@pytest.mark.parametrize("q_scale,latent_scale,swa_scale", [(2.0**40, 1.0, 1.0), (2.0**-40, 1.0, 1.0), (1.0, 100.0, 2.0**-30), (30.0, 1.0, 2.0**15),
                                                            (1.0, 2.0**-3, 2.0**-22), (1e-3, 1.0, 3e4)])
def test_attn_scales(lib, oracle_lib, q_scale, latent_scale, swa_scale):
    """Logits far apart, queries out of f16's range, windows whose records f16 cannot hold unscaled."""
    c = Case(oracle_lib, [700, 40], 64, seed=33, latent_scale=latent_scale, swa_scale=swa_scale)
    q = _decode_queries([700, 40]) + [(1, 0, 5, 3, 128)]
    c.check(lib, q, q_scale=q_scale, lse=abs(np.log2(q_scale)) < 10)
    assert lib.csa2_get_device_status() == 0


def test_attn_rising_logits(lib, oracle_lib):
    """A row whose later entries exceed every earlier maximum by far more than the lazy reference allows."""
    c = Case(oracle_lib, [1500], 64, seed=40)
    q = [(0, 1500, 1499, 92, 128)]
    c.run(lib, q)
    k = R.kv_values(R.paged_rows(c.pages, c.table[0], 64, range(1500)))
    # records reordered so that head 0's logits ascend, for a query large enough that they span hundreds
    order = np.argsort(k @ R.bf16_values(c.q[0, 0]).astype(np.float64))
    rec = R.paged_rows(c.pages, c.table[0], 64, order)
    for j in range(1500):
        c.pages[c.table[0, j // 64], j % 64] = rec[j]
    for s in (1.0, 16.0, 64.0):
        c.check(lib, q, q_scale=s, lse=s == 1.0)


def test_attn_same_bits_every_call(lib, oracle_lib):
    c = Case(oracle_lib, [4000, 17, 900], 64, seed=50)
    q = _decode_queries([4000, 17, 900])
    a, la = c.run(lib, q, fill=0x00)
    for fill in (0xFF, 0x7F, 0x3C):
        b, lb = c.run(lib, q, fill=fill)
        assert np.array_equal(a, b) and np.array_equal(la, lb)


def test_attn_out_of_range(lib, oracle_lib):
    c = Case(oracle_lib, [600, 200], 64, seed=60)
    good = (0, 600, 599, 0, 128)
    cap = c.table.shape[1] * 64
    for bad in [(2, 10, 0, 0, 0), (-1, 10, 0, 0, 0), (0, -1, 0, 0, 0), (0, cap + 1, 0, 0, 0), (0, 10, 0, 0, 129), (0, 10, 0, 128, 5),
                (0, 10, 0, -1, 5), (0, 10, 0, 0, -1)]:
        out, lse = c.run(lib, [good, bad, good])
        assert lib.csa2_get_device_status() == BOUNDS, bad
        assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))
        o, le, room = c.want([good], 0)
        assert row_norm_err(out[0], o) <= ATTN_TOL_F32
    # pages that do not exist: their entries are left out
    t = c.table.copy()
    t[0, 1], t[0, 4] = -1, c.n_pages
    c.check(lib, [good, (1, 200, 199, 0, 0)], table=t)
    assert lib.csa2_get_device_status() == BOUNDS
    # a selection that reaches behind the visible entries
    sel = np.array([[5, 599, 600, 2**31 - 1]])
    c.check(lib, [good], sel=sel)
    assert lib.csa2_get_device_status() == BOUNDS


def test_attn_lse_joins_disjoint_parts(lib, oracle_lib):
    """Outputs over two halves of the cache, joined by their lse, are the output over all of it."""
    from compressed_sparse_attention_index_gb300.shard import lse_merge
    c = Case(oracle_lib, [1000], 50, seed=70)
    whole, _ = c.run(lib, [(0, 1000, 999, 0, 0)])
    head, lh = c.run(lib, [(0, 500, 999, 0, 0)])
    t = c.table[:, 10:].copy()
    tail, lt = c.run(lib, [(0, 500, 999, 0, 0)], table=t)
    joined = lse_merge(np.stack([head[0], tail[0]]), np.stack([lh[0], lt[0]]))
    assert row_norm_err(joined, whole[0]) <= 2 * ATTN_TOL_F32


def test_attn_many_short_rows(lib, oracle_lib):
    """More rows than SMs: whole rows within a CTA, cut rows at its borders."""
    lens = [int(x) for x in np.random.default_rng(8).integers(0, 400, 330)]
    c = Case(oracle_lib, lens, 16, seed=80)
    q = _decode_queries(lens)
    out, lse = c.run(lib, q)
    for i in range(0, 330, 7):
        o, le, room = c.want(q, i)
        assert row_norm_err(out[i], o) <= ATTN_TOL_F32, i
    assert lib.csa2_get_device_status() == 0
