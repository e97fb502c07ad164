"""GPU tests of the operators that decide what a paged cache keeps at the calls that their contracts allow and ordinary
steps do not make: lengths far out of range, ranges that cross, runs long enough for every buffer to be used again."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import keep_reference as K  # noqa: E402
from tests.test_gpu_keep import BOUNDS, _i32, _tables  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


# ------------------------------------------------------------------ eviction
def _evict_told(lib, r, lens, told, keep, recent, page, in_place):
    """An eviction of sequences that have `lens` entries and are said to have `told`: (what the kernels leave, what they
    should, the bytes behind the workspace's declared size)."""
    n_seq, cols = len(lens), max(-(-n // page) for n in lens) + 1
    n_pages = sum(-(-n // page) for n in lens) + 2
    table, _ = _tables(r, lens, page, cols, n_pages)
    kept = [max(0, min(a, k)) for a, k in zip(lens, keep)]
    dst_cols, n_dst = max(1, max(-(-k // page) for k in kept)), sum(-(-k // page) for k in kept) + 2
    dst_table, _ = _tables(r, kept, page, dst_cols, n_dst)
    pages = r.integers(0, 256, (n_pages, page, 288), dtype=np.uint8)
    w = np.exp(2 * r.normal(size=n_pages * page)).astype(np.float32)
    P, W, T, L = torch.from_numpy(pages.copy()).cuda(), torch.from_numpy(w.copy()).cuda(), _i32(table), _i32(told)
    dP, dW, dT = torch.zeros((n_dst, page, 288), dtype=torch.uint8, device="cuda"), torch.zeros(n_dst * page, device="cuda"), _i32(dst_table)
    size = lib.csa2_workspace_size(lib.CSA2_OP_EVICT, n_seq, cols * page)
    ws = torch.full((size + (80 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    if in_place:
        lib.csa2_evict(P, W, n_pages, page, T, cols, L, _i32(keep), n_seq, recent, P, W, n_pages, T, cols, L, None, 0, ws, size)
    else:
        lib.csa2_evict(P, W, n_pages, page, T, cols, L, _i32(keep), n_seq, recent, dP, dW, n_dst, dT, dst_cols, L, None, 0, ws, size)
    status = lib.csa2_get_device_status()
    want = K.evict(pages, w, page, table, told, keep, recent, np.zeros_like(dP.cpu().numpy()), np.zeros(n_dst * page, np.float32),
                   table if in_place else dst_table, None, in_place)
    assert np.array_equal(L.cpu().numpy(), want[2])
    assert np.array_equal((P if in_place else dP).cpu().numpy(), want[0])
    assert np.array_equal((W if in_place else dW).cpu().numpy(), want[1].astype(np.float32))
    assert status == (0 if want[4] else BOUNDS)
    assert bool((ws[size:] == 0xA5).all())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("told", [{0: 90_000}, {4: 30_000}, {0: 2**31 - 1}, {4: 2**31 - 1}, {2: -1000}, {0: -(2**31)},
                                  {0: -5000, 1: 2**31 - 1, 3: -129}])
def test_evict_lengths_far_out_of_range(lib, in_place, told):
    """A sequence of an impossible length is left as it is, the others move, and nothing behind the workspace is written
    (its tiles were taken from the length that it was told)."""
    lens = [400, 700, 130, 1000, 260]
    _evict_told(lib, np.random.default_rng(len(told) + in_place), lens, [told.get(b, n) for b, n in enumerate(lens)],
                [150, 300, 70, 999, 5], 10, 16, in_place)


# ------------------------------------------------------------------ attention weights
def test_weigh_selections_of_refused_drafts():
    """plan, write, attend(sel), accept, weigh(sel), as a step is documented: refused drafts and rows without a token, whose
    selections still name entries, vote for nothing and are no error."""
    import compressed_sparse_attention_index_gb300 as lib
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    g = torch.Generator().manual_seed(4)
    rows = lambda n: (torch.randn((n, 64, 512), generator=g).bfloat16().cuda(), torch.randn((n, 512), generator=g).bfloat16().cuda())
    c = PagedCache(3, 90, 16, 400, 160, voters=20)
    c.step(_i32([90, 1, 69]), *rows(160))
    new, kept, k = [5, 4, 6], [2, 0, 6], 33
    for step in range(2):
        lens = c.seq_len.tolist()
        n = sum(new) + 3
        c.plan(_i32(new), rows=n)
        q, latent = rows(n)
        c.write(q, latent)
        sel = np.full((n, k), -1)
        at = 0
        for b in range(3):
            for t in range(new[b]):
                js = np.sort(np.random.default_rng(at + 50 * step).permutation(lens[b] + t + 1)[:k])
                sel[at, :len(js)] = js
                at += 1
        sel[at:] = np.arange(k)
        c.attend(_i32(sel))
        c.accept(_i32(kept))
        assert lib.csa2_get_device_status() == 0
        before = c.weight.cpu().numpy()
        c.weigh(_i32(sel), decay=0.5)
        status = lib.csa2_get_device_status()
        first, n_vis = np.concatenate([[0], np.cumsum(new)]), np.zeros(n, np.int64)
        for b in range(3):
            n_vis[first[b]:first[b] + kept[b]] = lens[b] + 1 + np.arange(kept[b])
        want, room, fine = K.attn_weight(c.q[:n].double().cpu().numpy(), c.pages.cpu().numpy(), 16, c.table.cpu().numpy(), first,
                                         np.where(n_vis[:, None] > 0, sel, -1), n_vis, c.lse[:n].cpu().numpy(), 0.5, before, before)
        assert fine and np.all(np.abs(c.weight.cpu().numpy() - want) <= room)
        assert status == 0


# ------------------------------------------------------------------ clusters
def test_clusters_beside_other_work(lib):
    """Rows that clusters share, verified and evicted while another stream's kernels hold SMs, so that the CTAs of a cluster
    do not find the chip empty: what they give alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    n_seq, vocab, n, page = 24, 131_072, 60_000, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = 3 * n_seq
    target = torch.softmax(2.5 * torch.randn((rows, vocab), generator=g, device="cuda"), 1)
    draft = torch.softmax(torch.log(target) + 0.5 * torch.randn((rows, vocab), generator=g, device="cuda"), 1)
    tokens = torch.randint(0, vocab, (rows,), generator=g, **i32)
    u, v = torch.rand(rows, generator=g, device="cuda") * 0.3, torch.rand(n_seq, generator=g, device="cuda")
    first = torch.arange(n_seq + 1, **i32) * 3
    cols = n // page
    table = torch.randperm(n_seq * cols, generator=g, device="cuda").to(torch.int32).view(n_seq, cols)
    pages = torch.randint(0, 256, (n_seq * cols, page, 288), generator=g, dtype=torch.uint8, device="cuda")
    weight = torch.rand(n_seq * n, generator=g, device="cuda")
    lens = torch.full((n_seq,), n, **i32)
    # all stay; the latest alone; some of both
    keeps = [(lens, 100), (lens // 2, n), (lens // 2, 500)]
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_EVICT, n_seq, n), dtype=torch.uint8, device="cuda")

    def call(stream):
        out = []
        for d in (draft, None):
            kept, nxt = torch.full((n_seq,), -5, **i32), torch.full((n_seq,), -5, **i32)
            lib.csa2_verify_drafts(lib.CSA2_VERIFY_SAMPLE, target, vocab, d, vocab if d is not None else 0, lib.CSA2_PROB_F32, vocab, tokens, first,
                                   n_seq, rows, u, v, kept, nxt, None, 0, stream)
            out += [kept, nxt]
        for keep, recent in keeps:
            dst, w, new = torch.zeros_like(pages), torch.zeros_like(weight), torch.zeros(n_seq, **i32)
            source = torch.full((n_seq, n), -1, **i32)
            lib.csa2_evict(pages, weight, len(pages), page, table, cols, lens, keep, n_seq, recent, dst, w, len(pages), table.flip(0).contiguous(), cols,
                           new, source, n, ws, ws.numel(), stream)
            out += [source, w, new]
        return out
    want = call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert all((want[4 + 3 * i][:, :k] >= 0).all() for i, k in ((0, n), (1, n // 2), (2, n // 2)))
    assert torch.equal(want[4], torch.arange(n, **i32).expand(n_seq, n)) and torch.equal(want[7][:, :n // 2], torch.arange(n - n // 2, n, **i32).expand(n_seq, -1))
    side, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    for _ in range(4):
        with torch.cuda.stream(side):
            b = a
            for _ in range(20):
                b = torch.sin(b @ a)
        got = call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert lib.csa2_get_device_status() == 0


def test_weigh_ranges_that_cross(lib):
    """Ranges of queries that descend and cross: whose work passes 32 bits, nothing is weighed and the error recorded."""
    page, stride, n_q, n_seq = 1 << 20, 2000, 60, 12             # 30 groups of two over 16 M chunks, from six of the ranges
    pages, w = torch.zeros((1, page, 288), dtype=torch.uint8, device="cuda"), torch.full((page,), -7.0, device="cuda")
    table = torch.zeros((n_seq, stride), dtype=torch.int32, device="cuda")
    q, lse = torch.ones((n_q, 64, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((n_q, 64), device="cuda")
    n_vis = torch.full((n_q,), page * stride, dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, n_q, n_seq, 0), dtype=torch.uint8, device="cuda")
    first = [0, n_q] * (n_seq // 2) + [n_q]
    lib.csa2_attn_weight(q, pages, 1, page, table, stride, _i32(first), n_seq, None, 0, n_vis, lse, n_q, 1.0, None, w, None, ws, ws.numel())
    assert lib.csa2_get_device_status() == BOUNDS
    assert bool((w == -7.0).all())


@pytest.mark.parametrize("first", [[0, 2, 100, 4, 6], [0, 2, -7, 4, 6], [0, 2, 1, 6, 6], [6, 0, 2, 2, 5]])
def test_weigh_selections_beside_a_range_that_is_out(lib, oracle_lib, first):
    """A range that is out of range takes its own sequence out, and no other, also where it stands in the way of a search."""
    from tests import paged_reference as R
    from tests.test_gpu_keep import _weigh, _weigh_case
    c = _weigh_case(oracle_lib, 21, [300, 200, 150, 400], 16, [2, 1, 1, 2], 40)
    c["first"] = np.array(first)
    c["n_vis"][:] = 140
    r = np.random.default_rng(1)
    c["sel"] = np.stack([np.sort(r.permutation(140)[:40]) for _ in range(6)])
    args = [R.bf16_values(c["q"]).astype(np.float64), c["pages"], 16, c["table"]]
    tail = [c["lse"], c["decay"], c["prior"], np.full(len(c["pages"]) * 16, -7.0)]
    # a query that two ranges have is one of theirs: here the one that a search of the starts comes upon, else the first
    valid = [b for b in range(4) if 0 <= first[b] <= first[b + 1] <= 6]
    owner = [[b for b in valid if first[b] <= i < first[b + 1]] for i in range(6)]
    got = _weigh(lib, c)
    status = lib.csa2_get_device_status()
    got = got.cpu().numpy()
    fits = []
    for pick in (0, -1):
        sel = []
        for b in range(4):                                    # one sequence at a time, the others' queries without a selection
            mine = np.array([bool(o) and o[pick] == b for o in owner])
            sel.append(np.where(mine[:, None], c["sel"], -1))
        want, room = tail[3].copy(), np.zeros(len(got))
        for b in valid:
            f = np.array([first[b], first[b + 1]])
            x, e, _ = K.attn_weight(*args[:3], args[3][b:b + 1], f, sel[b], c["n_vis"], *tail)
            touched = (x != -7.0) | (e > 0)
            want[touched], room[touched] = x[touched], e[touched]
        fits.append(bool(np.all(np.abs(got - want) <= room)))
    assert any(fits) and status == BOUNDS


def test_weigh_and_evict_behind_a_replayed_step():
    """A graph that holds a step up to accept; weigh and evict behind each replay, on the host's stream: the eager state."""
    import compressed_sparse_attention_index_gb300 as lib
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    from tests.test_gpu_keep_run import _state, _step_inputs
    new, keep = _i32([4, 3]), _i32([60, 1000])
    eager, graph = (PagedCache(2, 60, 16, 400, 100, voters=8) for _ in range(2))
    x = _step_inputs(3, 7)

    def step(c):
        c.plan(new, rows=7)
        c.write(x["q"], x["latent"])
        c.attend()
        c.verify(x["tokens"], x["target"], x["draft"], x["u"], x["v"])
        c.accept()
    for c in (eager, graph):
        c.step(_i32([60, 37]), *(_step_inputs(1, 97)[k] for k in ("q", "latent")))
        step(c)
        c.weigh(decay=0.5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graph)
    for seed in range(4, 8):
        for k, v in _step_inputs(seed, 7).items():
            x[k].copy_(v)
        step(eager)
        g.replay()
        for c in (eager, graph):
            c.weigh(decay=0.5, stream=torch.cuda.current_stream())
            if seed % 2 == 0:
                c.evict(keep, 20)
        a, b = _state(eager), _state(graph)
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), (seed, k)
    with pytest.raises(ValueError):
        eager.weigh()
    assert eager.gone[0] > 0 and lib.csa2_get_device_status() == 0


def test_evict_of_a_cache_says_which_entries_stayed():
    """What a caller keeps by place moves along by `source`; a sequence that it cannot hold stays."""
    import compressed_sparse_attention_index_gb300 as lib
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    g = torch.Generator().manual_seed(7)
    c = PagedCache(3, 60, 16, 300, 240, voters=240)
    c.step(_i32([150, 20, 70]), torch.randn((240, 64, 512), generator=g).bfloat16().cuda(), torch.randn((240, 512), generator=g).bfloat16().cuda())
    c.weigh()
    slot = lambda b, j: c.table[b].long()[j // 16] * 16 + j % 16
    was = [c.pages.view(-1, 288)[slot(b, torch.arange(n, device="cuda"))] for b, n in enumerate((150, 20, 70))]
    w = [c.weight[slot(b, torch.arange(n, device="cuda"))] for b, n in enumerate((150, 20, 70))]
    source = torch.full((3, 61), -9, dtype=torch.int32, device="cuda")
    c.evict(_i32([60, 30, 5]), 10, source=source)
    assert c.seq_len.tolist() == [60, 20, 5] and c.gone.tolist() == [90, 0, 65]
    for b, n in enumerate((60, 20, 5)):
        j = source[b, :n].long()
        assert torch.equal(c.pages.view(-1, 288)[slot(b, torch.arange(n, device="cuda"))], was[b][j]) and bool((j[1:] > j[:-1]).all())
        assert torch.equal(c.weight[slot(b, torch.arange(n, device="cuda"))], w[b][j]) and bool((source[b, n:] == -9).all())
    assert lib.csa2_get_device_status() == 0
    few = torch.full((3, 10), -9, dtype=torch.int32, device="cuda")
    c.evict(_i32([40, 9, 5]), 10, source=few)
    assert c.seq_len.tolist() == [60, 9, 5] and lib.csa2_get_device_status() == BOUNDS
    assert bool((few[0] == -9).all()) and few[2, :5].tolist() == [0, 1, 2, 3, 4]
