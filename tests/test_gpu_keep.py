"""GPU parity of the operators that decide what a paged cache keeps against their 64-bit restatements
(tests/keep_reference.py), through the C ABI: integers and moved bytes exactly, weights within the bound of
their fp32 sums."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gen import inputs as G  # noqa: E402
from tests import keep_reference as K  # noqa: E402
from tests import paged_reference as R  # noqa: E402

BOUNDS = 4


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


def _i32(x):
    return torch.from_numpy(np.array(x, np.int32)).cuda()


def _f32(x):
    return torch.from_numpy(np.array(x, np.float32)).cuda()


def _bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _records(oracle_lib, n, seed):
    return oracle_lib.pack_kv(G.normal_block_bf16(seed, G.S_LATENT, 3, 0, n, 512))


def _tables(r, lens, page, cols, n_pages):
    table = np.full((len(lens), cols), -1, np.int64)
    ids, k = r.permutation(n_pages), 0
    for b, n in enumerate(lens):
        have = -(-int(n) // page)
        table[b, :have] = ids[k:k + have]
        k += have
    return table, ids[k:]


# ------------------------------------------------------------------ attention weights
def _weigh_case(oracle_lib, seed, lens, page, counts, sel=0, spare=2):
    """Sequences of these lengths with so many queries each: query t of G sees up to itself."""
    r = np.random.default_rng(seed)
    cols = max(1, max(-(-n // page) for n in lens))
    n_pages = sum(-(-n // page) for n in lens) + spare
    table, _ = _tables(r, lens, page, cols, n_pages)
    pages = _records(oracle_lib, n_pages * page, seed).reshape(n_pages, page, 288)
    n_q = sum(counts)
    c = dict(pages=pages, page=page, table=table, first=np.concatenate([[0], np.cumsum(counts)]),
             q=G.normal_block_bf16(seed, G.S_Q, 5, 0, n_q * 64, 512).reshape(n_q, 64, 512), sel=None,
             n_vis=np.array([max(0, n - g + t + 1) for n, g in zip(lens, counts) for t in range(g)], np.int64),
             decay=0.75, prior=r.exponential(size=n_pages * page).astype(np.float32))
    seen = np.maximum(1, np.minimum(c["n_vis"], sel) if sel else c["n_vis"])
    c["lse"] = (np.log(seen + 60.0)[:, None] + 0.5 + 0.2 * r.normal(size=(n_q, 64))).astype(np.float32)
    if sel:
        c["sel"] = np.full((n_q, sel), -1, np.int64)
        for i, v in enumerate(c["n_vis"]):
            js = np.sort(r.permutation(v)[:sel])
            c["sel"][i, :len(js)] = js
    return c


def _weigh(lib, c, stream=None, out=None):
    n_pages, n_q, n_seq = len(c["pages"]), len(c["q"]), len(c["first"]) - 1
    d = c.setdefault("_dev", {})
    if not d:
        d.update(q=_bf16(c["q"]), pages=torch.from_numpy(np.ascontiguousarray(c["pages"])).cuda(), table=_i32(c["table"]),
                 first=_i32(c["first"]), sel=None if c["sel"] is None else _i32(c["sel"]), n_vis=_i32(c["n_vis"]),
                 lse=_f32(c["lse"]), prior=None if c["prior"] is None else _f32(c["prior"]))
    k = 0 if c["sel"] is None else c["sel"].shape[1]
    w = torch.full((n_pages * c["page"],), -7.0, device="cuda") if out is None else out
    ws = torch.full((lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, n_q, n_seq, k),), 0xA5, dtype=torch.uint8, device="cuda")
    lib.csa2_attn_weight(d["q"], d["pages"], n_pages, c["page"], d["table"], c["table"].shape[1], d["first"], n_seq,
                         d["sel"], k, d["n_vis"], d["lse"], n_q, c["decay"], d["prior"], w, None, ws, ws.numel(), stream)
    return w


def _check_weigh(lib, c):
    got = _weigh(lib, c)
    status = lib.csa2_get_device_status()
    want, room, fine = K.attn_weight(R.bf16_values(c["q"]).astype(np.float64), c["pages"], c["page"], c["table"], c["first"],
                                     c["sel"], c["n_vis"], c["lse"], c["decay"], c["prior"], np.full(got.numel(), -7.0))
    got = got.cpu().numpy().astype(np.float64)
    assert status == (0 if fine else BOUNDS)
    assert np.array_equal(got[room == 0], want[room == 0])           # untouched, or the prior alone
    assert np.all(np.abs(got - want) <= room), float(np.max(np.abs(got - want) / np.maximum(room, 1e-300)))
    return got, want


@pytest.mark.parametrize("lens,page,counts", [
    ([1], 64, [1]), ([1, 2, 3], 1, [1, 2, 3]), ([127, 128, 129], 16, [1, 2, 3]), ([257, 0, 31], 7, [5, 0, 1]),
    ([640, 100, 5], 48, [1, 6, 4]), ([300, 1000], 100, [17, 1]), ([2500], 64, [1]), ([900] * 9, 128, [2] * 9),
    ([3, 3, 260], 4, [3, 1, 9])])
def test_weights(lib, oracle_lib, lens, page, counts):
    _check_weigh(lib, _weigh_case(oracle_lib, 10 + len(lens) + page, lens, page, counts))


@pytest.mark.parametrize("lens,page,counts,sel", [([700], 64, [1], 512), ([1, 130], 16, [1, 2], 1), ([400, 90, 2000], 48, [5, 3, 1], 77),
                                                  ([600], 1, [8], 300), ([64, 64], 7, [0, 2], 512)])
def test_weights_of_selections(lib, oracle_lib, lens, page, counts, sel):
    _check_weigh(lib, _weigh_case(oracle_lib, 40 + sel, lens, page, counts, sel))


@pytest.mark.parametrize("sel", [0, 100])
def test_weights_prior_and_decay(lib, oracle_lib, sel):
    for decay, prior in ((0.0, "other"), (1.0, "other"), (1.0, None), (0.5, "own"), (1.0, "own"), (-1.0, "own")):
        c = _weigh_case(oracle_lib, 77, [400, 333], 16, [2, 1], sel)
        c["decay"] = decay
        if prior is None:
            c["prior"] = None
        if prior == "own":                               # in place: slots of no entry keep their prior
            _weigh(lib, c)
            w = c["_dev"]["prior"]
            want, room, _ = K.attn_weight(R.bf16_values(c["q"]).astype(np.float64), c["pages"], c["page"], c["table"],
                                          c["first"], c["sel"], c["n_vis"], c["lse"], decay, c["prior"], c["prior"])
            _weigh(lib, c, out=w)
            assert np.all(np.abs(w.cpu().numpy() - want) <= room)
        else:
            _check_weigh(lib, c)
    assert lib.csa2_get_device_status() == 0


def test_weights_of_attention_add_up(lib, oracle_lib):
    """With csa2_paged_attn's own log-sum-exp and no window a query gives its 64 heads' weights away: 64 in all."""
    c = _weigh_case(oracle_lib, 5, [1500, 70], 32, [3, 2])
    c["prior"] = None
    n_q, z = 5, _i32(np.zeros(5))
    lse, out = torch.empty((n_q, 64), device="cuda"), torch.empty((n_q, 64, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, n_q, 0), dtype=torch.uint8, device="cuda")
    pages, table = torch.from_numpy(c["pages"]).cuda(), _i32(c["table"])
    lib.csa2_paged_attn(_bf16(c["q"]), pages, len(c["pages"]), 32, table, c["table"].shape[1], 2, None, 0, None, 0,
                        _i32([0, 0, 0, 1, 1]), _i32(c["n_vis"]), _i32(c["n_vis"] - 1), z, z, n_q, out,
                        lib.CSA2_OUT_BF16, lse, None, ws, ws.numel())
    c["lse"] = lse.cpu().numpy()
    got, _ = _check_weigh(lib, c)
    # 1,570 entries' errors, each 2^-15 of its weight and about as much of the log-sum-exp's
    assert abs(got[got != -7.0].sum() - 64 * n_q) < 64 * n_q * 2.0**-12


def test_weights_out_of_range(lib, oracle_lib):
    c = _weigh_case(oracle_lib, 8, [300, 200, 150], 16, [2, 2, 2])
    c["n_vis"][1], c["n_vis"][2] = -3, c["table"].shape[1] * 16 + 1
    c["table"][2, 3], c["table"][0, 5] = -1, len(c["pages"])
    _check_weigh(lib, c)
    for first in ([0, 2, 1, 6], [-1, 2, 4, 6], [0, 2, 4, 7]):
        c = _weigh_case(oracle_lib, 8, [300, 200, 150], 16, [2, 2, 2])
        c["first"] = np.array(first)
        _check_weigh(lib, c)
    c = _weigh_case(oracle_lib, 9, [300, 200], 16, [2, 2], 40)
    c["sel"][0, 7], c["sel"][1, 9], c["sel"][3, :] = 299, 2**31 - 1, -1        # (query 0 sees 299 entries)
    c["sel"][2, 3] = c["sel"][2, 4] = c["sel"][2, 30]                           # named three times
    c["table"][0, 3] = -1
    _check_weigh(lib, c)


def test_weights_heads_that_are_not_finite_or_large(lib, oracle_lib):
    c = _weigh_case(oracle_lib, 12, [290], 16, [3])
    q = R.bf16_values(c["q"]).copy()
    q[0, 3, 7], q[0, 4, 8], q[1, 5, :] = np.nan, np.inf, 0.0
    q[1, 6] *= 2.0**100
    q[1, 7] *= 2.0**-100
    q[2, 8] *= 2.0**-20
    q[2, 9, 5] *= 2.0**24                                 # one element far above the head's others
    c["q"] = R.round_bf16_bits(np.nan_to_num(q, nan=1.0, posinf=1.0).astype(np.float64))
    c["q"][0, 3, 7], c["q"][0, 4, 8] = 0x7FC0, 0x7F80
    c["lse"][0, 10:13] = [np.nan, np.inf, -np.inf]
    # lse of the large heads as attention would return them
    k = R.kv_values(np.concatenate([c["pages"][p] for p in c["table"][0]])[:290])
    for i, h in ((1, 6), (2, 9)):
        logit = 512 ** -0.5 * (k[:c["n_vis"][i]] @ R.bf16_values(c["q"][i, h]).astype(np.float64))
        c["lse"][i, h] = logit.max() + 1.0
    _check_weigh(lib, c)


def test_weights_of_heads_of_unlike_size(lib, oracle_lib):
    """Heads and elements of other sizes whose logits fp32 still knows to a few per mille; heads that add nothing."""
    c = _weigh_case(oracle_lib, 13, [290, 140], 16, [3, 1])
    q = R.bf16_values(c["q"]).copy()
    q[0, 5], q[0, 6] = 0.0, q[0, 6] * 2.0**-100
    q[1, 7] *= 2.0**4
    q[1, 8] *= 2.0**-20
    q[2, 9, 5] *= 2.0**6
    q[2, 10, 1:] *= 2.0**-24
    q[3] *= 2.0**-130
    c["q"] = R.round_bf16_bits(q.astype(np.float64))
    c["q"][0, 3, 7], c["q"][0, 4, 8], c["q"][2, 60, 511] = 0x7FC0, 0x7F80, 0xFF80
    c["lse"][0, 10:13] = [np.nan, np.inf, -np.inf]
    c["lse"][1, 7], c["lse"][2, 9] = 60.0, 30.0
    got, want = _check_weigh(lib, c)
    assert np.all(np.isfinite(want))


def test_weights_far_in_a_large_cache(lib, oracle_lib):
    """Slots beyond 4 GiB of records."""
    page, n_pages = 1 << 16, 236                         # 15.5 M records, 4.45 GB
    pages = torch.zeros((n_pages, page, 288), dtype=torch.uint8, device="cuda")
    rec = _records(oracle_lib, 400, 3)
    pages[n_pages - 1, :400] = torch.from_numpy(rec).cuda()
    w = torch.zeros(n_pages * page, device="cuda")
    q = G.normal_block_bf16(3, G.S_Q, 5, 0, 64, 512).reshape(1, 64, 512)
    lse = np.full((1, 64), 6.0, np.float32)
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, 1, 1, 0), dtype=torch.uint8, device="cuda")
    lib.csa2_attn_weight(_bf16(q), pages, n_pages, page, _i32([[n_pages - 1]]), 1, _i32([0, 1]), 1, None, 0, _i32([400]),
                         _f32(lse), 1, 1.0, None, w, None, ws, ws.numel())
    assert lib.csa2_get_device_status() == 0
    want, room, _ = K.attn_weight(R.bf16_values(q).astype(np.float64), rec[None], 400, np.array([[0]]), [0, 1], None, [400], lse,
                                  1.0, None, np.zeros(400))
    got = w.cpu().numpy()
    assert np.all(np.abs(got[-page:][:400] - want) <= room) and not got[:-page].any() and not got[-page + 400:].any()
    # and moved back within the page
    keep = torch.empty(1, dtype=torch.int32, device="cuda")
    t = _i32([[n_pages - 1]])
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_EVICT, 1, page), dtype=torch.uint8, device="cuda")
    lib.csa2_evict(pages, w, n_pages, page, t, 1, _i32([400]), _i32([100]), 1, 7, pages, w, n_pages, t, 1, keep, None, 0, ws, ws.numel())
    assert lib.csa2_get_device_status() == 0 and keep.tolist() == [100]
    stay = sorted(sorted(range(393), key=lambda j: (-got[-page + j], j))[:93]) + list(range(393, 400))
    assert np.array_equal(pages[n_pages - 1, :100].cpu().numpy(), rec[stay])


def test_weights_far_in_a_long_row(lib, oracle_lib):
    """A row of nearly 2^31 places, most of them without a page; selected entries at its end, and one behind it."""
    page = 1 << 20
    stride = (2**31 - 256) // page
    n = stride * page
    table = np.full((1, stride), -1)
    table[0, -1] = 1
    pages = torch.zeros((2, page, 288), dtype=torch.uint8, device="cuda")
    rec = _records(oracle_lib, 300, 5)
    pages[1, page - 300:] = torch.from_numpy(rec).cuda()
    w = torch.full((2 * page,), -7.0, device="cuda")
    q = G.normal_block_bf16(3, G.S_Q, 5, 0, 64, 512).reshape(1, 64, 512)
    lse = np.full((1, 64), 3.0, np.float32)
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, 1, 1, 5), dtype=torch.uint8, device="cuda")
    lib.csa2_attn_weight(_bf16(q), pages, 2, page, _i32(table), stride, _i32([0, 1]), 1, _i32([[n - 1, n - 2, n - 300, n, -1]]), 5,
                         _i32([n]), _f32(lse), 1, 1.0, w, w, None, ws, ws.numel())
    assert lib.csa2_get_device_status() == BOUNDS
    k = R.kv_values(rec[[299, 298, 0]])
    x = 512 ** -0.5 * (k @ R.bf16_values(q)[0].astype(np.float64).T) - 3.0
    got = w.cpu().numpy()
    at = page + np.array([page - 1, page - 2, page - 300])
    # fp32 sums of 512 products of magnitudes that add up to about 15 (2^-14 of them), and the sum with -7
    assert np.all(np.abs(got[at] + 7.0 - np.exp(x).sum(1)) <= 2.0**-9 * np.exp(x).sum(1) + 2.0**-20)
    assert np.count_nonzero(got != -7.0) == 3


# ------------------------------------------------------------------ eviction
def _evict(lib, seed, lens, keep, recent, page, in_place, weights="random", want_from=True, spoil=None):
    r = np.random.default_rng(seed)
    n_seq = len(lens)
    cols = max(1, max(-(-int(n) // page) for n in lens)) + 1
    n_pages = sum(-(-int(n) // page) for n in lens) + 2
    table, _ = _tables(r, lens, page, cols, n_pages)
    pages = r.integers(0, 256, (n_pages, page, 288), dtype=np.uint8)
    n = n_pages * page
    w = {"random": lambda: np.exp(2 * r.normal(size=n)), "few": lambda: r.integers(0, 4, n) * 0.25, "same": lambda: np.full(n, 0.5),
         "odd": lambda: np.where(r.random(n) < 0.2, np.nan, np.where(r.random(n) < 0.3, r.choice([0.0, -0.0, -1.0, np.inf, -np.inf, 1e-40], n), r.normal(size=n)))}
    w = w[weights]().astype(np.float32)
    kept = [min(int(a), int(k)) for a, k in zip(lens, keep)]
    n_dst = sum(-(-max(k, 0) // page) for k in kept) + 2
    dst_cols = max(1, max(-(-max(k, 0) // page) for k in kept))
    dst_table, _ = _tables(r, [max(k, 0) for k in kept], page, dst_cols, n_dst)
    lens, keep = np.array(lens), np.array(keep)
    if spoil:
        spoil(lens, keep, table, dst_table)
    stride = dst_cols * page
    dev = lambda x: torch.from_numpy(np.array(x)).cuda()
    P, W, T, L = dev(pages), dev(w), _i32(table), _i32(lens)
    dP, dW = dev(np.full((n_dst, page, 288), 0xAB, np.uint8)), torch.full((n_dst * page,), -3.0, device="cuda")
    dT = _i32(dst_table)
    fr = torch.full((n_seq, stride), -1, dtype=torch.int32, device="cuda") if want_from else None
    new = torch.full((n_seq,), -9, dtype=torch.int32, device="cuda")
    ws = torch.full((lib.csa2_workspace_size(lib.CSA2_OP_EVICT, n_seq, cols * page),), 0xA5, dtype=torch.uint8, device="cuda")
    if in_place:
        new = L                                           # the lengths are replaced
        lib.csa2_evict(P, W, n_pages, page, T, cols, L, _i32(keep), n_seq, recent, P, W, n_pages, T, cols, new, fr, stride, ws, ws.numel())
    else:
        lib.csa2_evict(P, W, n_pages, page, T, cols, L, _i32(keep), n_seq, recent, dP, dW, n_dst, dT, dst_cols, new, fr, stride, ws, ws.numel())
    status = lib.csa2_get_device_status()
    want = K.evict(pages, w, page, table, lens, keep, recent, np.full((n_dst, page, 288), 0xAB, np.uint8),
                   np.full(n_dst * page, -3.0, np.float32), table if in_place else dst_table, stride if want_from else None, in_place)
    if want_from:
        rows = np.full((n_seq, stride), -1)
        for b, js in enumerate(want[3]):
            rows[b, :len(js)] = js
        assert np.array_equal(fr.cpu().numpy(), rows)
    assert np.array_equal(new.cpu().numpy(), want[2])
    assert np.array_equal((P if in_place else dP).cpu().numpy(), want[0])
    assert np.array_equal((W if in_place else dW).cpu().numpy().view(np.uint32), want[1].astype(np.float32).view(np.uint32))
    if not in_place:
        assert np.array_equal(P.cpu().numpy(), pages) and np.array_equal(W.cpu().numpy().view(np.uint32), w.view(np.uint32))
    assert status == (0 if want[4] else BOUNDS)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep,recent,page", [
    ([1], [1], 0, 64), ([1, 1, 5], [0, 1, 3], 1, 1), ([0, 300, 17], [5, 100, 17], 16, 16), ([127, 128, 129, 130], [64, 127, 128, 1], 3, 7),
    ([1000], [999], 0, 48), ([1000, 900], [1, 0], 5, 100), ([700, 50, 3000], [650, 60, 1500], 2000, 64), ([5000, 4097, 4096], [2500, 4096, 17], 128, 128),
    ([260] * 40, [131] * 40, 10, 32)])
def test_evict(lib, lens, keep, recent, page, in_place):
    for i, weights in enumerate(("random", "few", "odd")):
        _evict(lib, 100 * len(lens) + page + i, lens, keep, recent, page, in_place, weights, want_from=i != 1)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_rows(lib, in_place):
    """Rows that a cluster shares, in shared memory and, longer ones, out of L2; ties across its CTAs."""
    _evict(lib, 1, [60_000], [30_000], 100, 16, in_place)
    _evict(lib, 2, [200_001], [777], 0, 7, in_place, "few")
    _evict(lib, 3, [150_000, 9], [149_000, 9], 1, 64, in_place, "same", want_from=False)
    _evict(lib, 4, [1_000_003], [500_000], 4096, 100, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_seq,n,recent", [(1, 20_000, 0), (14, 30_000, 5), (9, 45_000, 0), (3, 110_003, 700), (8, 70_001, 0), (20, 24_000, 24_000)])
def test_evict_clusters_of_any_size(lib, n_seq, n, recent, in_place):
    """Rows that 3, 4, 6, 9 or more CTAs share: histograms that do not divide evenly among them."""
    r = np.random.default_rng(n)
    lens = [n] + r.integers(0, n + 1, n_seq - 1).tolist()
    keep = r.integers(1, n, n_seq).tolist()
    for weights in ("random", "odd"):
        _evict(lib, n_seq, lens, keep, recent, 32, in_place, weights, want_from=weights == "odd")


def test_evict_out_of_range(lib):
    def lengths(lens, keep, table, dst_table):
        lens[0], keep[1], lens[2] = -1, -5, table.shape[1] * 16 + 1
    def columns(lens, keep, table, dst_table):
        table[1, 2], table[0, 0] = -1, 10_000
        dst_table[3, 1] = -4
    def too_many(lens, keep, table, dst_table):
        keep[:] = 1000                                    # more than the destination's rows and from hold
    for in_place in (False, True):
        _evict(lib, 7, [200, 100, 150, 90], [80, 50, 20, 40], 4, 16, in_place, spoil=lengths)
        _evict(lib, 9, [200, 100, 150, 90], [80, 50, 20, 40], 4, 16, in_place, spoil=too_many)
    _evict(lib, 8, [200, 100, 150, 90], [80, 90, 20, 40], 4, 16, False, spoil=columns)
    _evict(lib, 8, [200, 100, 150, 90], [80, 90, 20, 40], 4, 16, True, spoil=lambda a, k, t, d: t.__setitem__((1, 2), -1))


# ------------------------------------------------------------------ pages given back
@pytest.mark.parametrize("n_seq,page,seed", [(1, 64, 0), (5, 1, 1), (300, 16, 2), (3000, 7, 3), (16384, 32, 4)])
def test_trim(lib, n_seq, page, seed):
    r = np.random.default_rng(seed)
    lens = r.integers(0, 5 * page, n_seq)
    to = (lens * r.random(n_seq)).astype(np.int64)
    cols = 6
    n_pages = int(sum(-(-lens // page))) + 9
    table, rest = _tables(r, lens, page, cols, n_pages)
    free = np.concatenate([r.permutation(n_pages - len(rest)), rest])
    head = n_pages - len(rest)
    for spoil in (False, True):
        if spoil:
            lens[0], to[n_seq // 2] = -2, lens[n_seq // 2] + 1
        F, H, T = _i32(free), _i32([head]), _i32(table)
        lib.csa2_page_trim(_i32(lens), _i32(to), n_seq, page, n_pages, F, n_pages, H, T, cols)
        want = K.trim(lens, to, page, n_pages, free, head, table)
        assert np.array_equal(F.cpu().numpy(), want[0]) and H.tolist() == [want[1]] and np.array_equal(T.cpu().numpy(), want[2])
        assert lib.csa2_get_device_status() == (0 if want[3] else BOUNDS)
    assert not want[3]


def test_trim_out_of_range(lib):
    for lens, to, head, table in (([64, 64], [0, 0], 1, [[1, 2], [3, 4]]), ([64], [0], -1, [[1, 2]]), ([64], [0], 9, [[1, 2]]),
                                  ([64], [0], 4, [[-1, 77]])):
        F, H, T = _i32([9, 8, 7, 6]), _i32([head]), _i32(table)
        lib.csa2_page_trim(_i32(lens), _i32(to), len(lens), 32, 10, F, 4, H, T, 2)
        want = K.trim(lens, to, 32, 10, [9, 8, 7, 6], head, table)
        assert F.tolist() == want[0].tolist() and H.tolist() == [want[1]] and T.tolist() == want[2].tolist()
        assert lib.csa2_get_device_status() == BOUNDS and not want[3]


# ------------------------------------------------------------------ verification
TYPES = {"f32": (torch.float32, "CSA2_PROB_F32"), "bf16": (torch.bfloat16, "CSA2_PROB_BF16"), "f16": (torch.float16, "CSA2_PROB_F16")}


def _verify(lib, kind, target, draft, vocab, tokens, first, u, v, greedy=False, pad=0, shift=0):
    """target, draft: fp64 [rows][vocab]; both sides get them rounded to `kind`."""
    dt, name = TYPES[kind]
    def rows(x, shift):
        if x is None:
            return None
        buf = torch.full((len(x) * (vocab + pad) + 16,), float("nan"), dtype=dt, device="cuda")
        view = buf[shift:shift + len(x) * (vocab + pad)].view(len(x), vocab + pad)
        view[:, :vocab] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)
        return view
    t, d = rows(target, shift), rows(draft, shift + (1 if pad % 2 else 0))
    n_seq, n_rows = len(first) - 1, len(target)
    kept, nxt = torch.full((n_seq,), -5, dtype=torch.int32, device="cuda"), torch.full((n_seq,), -5, dtype=torch.int32, device="cuda")
    ws = torch.full((max(1, lib.csa2_workspace_size(lib.CSA2_OP_VERIFY, n_rows, 0)),), 0xA5, dtype=torch.uint8, device="cuda")
    lib.csa2_verify_drafts(1 if greedy else 0, t, vocab + pad, d, vocab + pad, getattr(lib, name), vocab, _i32(tokens), _i32(first),
                           n_seq, n_rows, _f32(u), _f32(v), kept, nxt, ws, ws.numel())
    status = lib.csa2_get_device_status()
    f64 = lambda x: None if x is None else x[:, :vocab].double().cpu().numpy()
    want = K.verify(greedy, f64(t), f64(d), vocab, tokens, first, np.float32(u), np.float32(v))
    assert kept.tolist() == want[0].tolist() and nxt.tolist() == want[1].tolist()
    assert status == (0 if want[2] else BOUNDS)
    return want


def _softmax(x):
    x = np.exp(x - x.max(-1, keepdims=True))
    return x / x.sum(-1, keepdims=True)


def _verify_case(seed, counts, vocab, close=0.5):
    r = np.random.default_rng(seed)
    first, n = np.concatenate([[0], np.cumsum(counts)]), int(sum(counts))
    x = 2 * r.normal(size=(n, vocab))
    target, draft = _softmax(x), _softmax(x + close * r.normal(size=(n, vocab)))
    tokens = np.zeros(n, np.int64)
    for i in range(n - 1):
        tokens[i + 1] = min(vocab - 1, np.searchsorted(np.cumsum(draft[i]), r.random()))
    return target, draft, tokens, first, r.random(n).astype(np.float32), r.random(len(counts)).astype(np.float32)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,vocab,pad,shift", [([1], 1, 0, 0), ([4, 0, 2], 7, 0, 1), ([6], 1000, 3, 0), ([6, 1, 3, 2] * 5, 4099, 0, 3),
                                                    ([2, 6, 1], 32_003, 5, 2), ([6, 4], 131_072, 0, 0), ([70, 40], 300, 8, 0)])
def test_verify(lib, kind, counts, vocab, pad, shift):
    for seed in range(3):
        t, d, tok, first, u, v = _verify_case(seed + vocab, counts, vocab, 0.1 if max(counts) > 30 else 0.5)
        _verify(lib, kind, t, d, vocab, tok, first, u, v, pad=pad, shift=shift)
        _verify(lib, kind, t, None, vocab, tok, first, u * 0.01, v, pad=pad, shift=shift)
        best = np.concatenate([[0], t.argmax(1)[:-1]])
        _verify(lib, kind, np.log(t), None, vocab, np.where(np.random.default_rng(seed).random(len(tok)) < 0.7, best, tok), first, u, v, True, pad, shift)


def test_verify_decides_at_borders(lib):
    """Running sums that are exact multiples of 2^-k, and numbers on them: 'above' is above."""
    n = 1024
    flat = np.full((1, n), 2.0**-10)
    for j in (0, 1, 127, 128, 511, 1000, 1023):
        assert _verify(lib, "f32", flat, None, n, [0], [0, 1], [0.0], [j / n])[1] == [j]
        assert _verify(lib, "f32", flat, None, n, [0], [0, 1], [0.0], [np.nextafter(np.float32((j + 1) / n), np.float32(0))])[1] == [j]
    # a draft stays while u q < p: at equality it does not
    t, d = np.zeros((2, 8)), np.zeros((2, 8))
    t[0, 3], t[0, 5], d[0, 3], t[1, 6] = 0.25, 0.75, 0.5, 1.0
    assert _verify(lib, "f32", t, d, 8, [0, 3], [0, 2], [0.5, 0], [0.9])[0] == [1]
    assert _verify(lib, "f32", t, d, 8, [0, 3], [0, 2], [np.nextafter(np.float32(0.5), np.float32(0)), 0], [0.9])[0] == [2]
    # a large vocabulary of tiny probabilities beside one of nearly one: fp32 sums would lose them
    v = 100_000
    p = np.full((1, v), 2.0**-30)
    p[0, 0] = 1.0
    for j in (1, 2, 50_000, 99_998):
        goal = (1 + (j + 0.5) * 2.0**-30) / p.sum()
        got = _verify(lib, "f32", p, None, v, [0], [0, 1], [0.0], [goal])[1][0]
        assert got == 0 or abs(got - j) <= 2.0**-24 * 2.0**30    # (v itself is fp32; both sides agree to the token)


def test_verify_with_nothing_left(lib):
    t, d, tok, first, u, v = _verify_case(3, [3, 3, 2], 500)
    _verify(lib, "f32", t, t.copy(), 500, tok, first, np.full(8, 1.0), v)            # p - q is zero everywhere: p itself
    t[0:1], t[4] = 0.0, 0.0                                                          # no probability at all
    _verify(lib, "f32", t, d, 500, tok, first, u, v)
    t2 = t.copy()
    t2[1, :100], t2[2, 5], t2[3, 7], t2[5, :] = -0.5, np.nan, np.inf, np.nan
    d[0, 3], d[3, :50] = np.nan, -1.0
    _verify(lib, "f32", t2, d, 500, tok, first, u, v)
    _verify(lib, "f32", t2, None, 500, tok, first, u, v, True)                       # a row of NaN alone
    tok[1], tok[4] = 500, -1                                                         # drafts that are no tokens
    _verify(lib, "f32", np.abs(_softmax(np.random.default_rng(1).normal(size=(8, 500)))), d, 500, tok, first, u, v)
    _verify(lib, "bf16", t, None, 500, tok, first, u, v, True)


def test_verify_ends_of_the_numbers(lib):
    t, d, tok, first, u, v = _verify_case(9, [2, 1, 3], 3001)
    for x in (0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0):
        _verify(lib, "f32", t, d, 3001, tok, first, np.full(6, x), np.full(3, x))
        _verify(lib, "bf16", t, None, 3001, tok, first, np.full(6, x), np.full(3, x))


def test_verify_greedy_ties(lib):
    t = np.zeros((4, 700))
    t[0, [3, 600]], t[1, :], t[2, 10], t[2, 11] = 2.0, -np.inf, 0.0, -0.0
    t[2, :10], t[2, 12:] = -1.0, -1.0
    t[3, :] = np.arange(700) % 7
    assert _verify(lib, "f32", t, None, 700, [1, 3, 0, 10], [0, 4], [0] * 4, [0], True)[0] == [4]
    assert _verify(lib, "f32", t, None, 700, [1, 600, 0, 10], [0, 4], [0] * 4, [0], True)[1] == [3]


def test_verify_first_out_of_range(lib):
    t, d, tok, first, u, v = _verify_case(4, [2, 2, 2], 100)
    for bad in ([0, 2, 1, 6], [-1, 2, 4, 6], [0, 2, 4, 7]):
        _verify(lib, "f32", t, d, 100, tok, bad, u, v)


# ------------------------------------------------------------------ plan behind evictions
@pytest.mark.parametrize("n_seq,page,cap,seed", [(1, 64, 128, 0), (40, 16, 130, 1), (700, 7, 192, 2), (9, 48, 40, 3), (5, 16, 0, 4)])
def test_plan_at(lib, n_seq, page, cap, seed):
    r = np.random.default_rng(seed)
    ln, new, gone = r.integers(0, 500, n_seq), r.integers(0, 6, n_seq), r.integers(0, 2000, n_seq) * (r.random(n_seq) < 0.7)
    gone[-1] = 2**31 - 1 - ln[-1] - new[-1]
    cols, n_pages = -(-520 // page), n_seq * (-(-520 // page)) + 4
    table, rest = _tables(r, ln, page, cols, n_pages)
    m = int(new.sum()) + 3
    for spoil in (False, True):
        if spoil:
            gone[0] = -1 if n_seq > 1 else gone[0] + 1
        T, desc = _i32(table), torch.full((7, m), -77, dtype=torch.int32, device="cuda")
        first, totals = torch.empty(n_seq + 1, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
        lib.csa2_page_plan_at(_i32(ln), _i32(new), _i32(gone), n_seq, page, n_pages, _i32(rest), len(rest), None, T, cols, cap, desc, m, first, totals)
        keep = new.copy()
        if spoil:
            keep[0] = 0
        # places as without losses; positions, windows and ring slots further on
        want = R.plan(ln, keep, page, n_pages, rest, 0, table, cap, m)
        d = want[0].copy()
        for i in range(int(keep.sum())):
            b = d[0, i]
            pos = d[2, i] + gone[b]
            cnt = min(128, cap, pos + 1)
            d[2, i], d[4, i] = pos, cnt
            d[3, i] = (pos + 1 - cnt) % cap if cap else 0
            d[6, i] = b * cap + pos % cap if cap and pos + cap >= gone[b] + ln[b] + keep[b] else -1
        assert np.array_equal(desc.cpu().numpy(), d) and np.array_equal(T.cpu().numpy(), want[3])
        assert np.array_equal(first.cpu().numpy(), want[1]) and totals.tolist() == want[2].tolist()
        assert lib.csa2_get_device_status() == (BOUNDS if spoil else 0)
