"""The paged-cache operators run together, as a server runs them: steps of a
PagedCache against the plain restatement, captured and replayed, on other
streams, two at once; and attention calls that the single-operator tests leave
out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_reference as R  # noqa: E402
from parity import ATTN_TOL_BF16, ATTN_TOL_F32, row_norm_err  # noqa: E402
from test_gpu_paged import BOUNDS, Case, _bf16, _bits, _decode_queries, _i32  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


def _cache(n_seq, n_pages, page, max_len, max_tokens, cap=128, f32=True):
    import compressed_sparse_attention_index_gb300 as c
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    return PagedCache(n_seq, n_pages, page, max_len, max_tokens, cap, c.CSA2_OUT_F32 if f32 else c.CSA2_OUT_BF16)


def _inputs(m, seed):
    g = torch.Generator().manual_seed(seed)
    return (2 * torch.randn((m, 64, 512), generator=g)).bfloat16().cuda(), (3 * torch.randn((m, 512), generator=g)).bfloat16().cuda()


@pytest.mark.parametrize("page,cap", [(16, 260), (7, 300), (64, 256)])
def test_steps_against_the_plain_restatement(lib, oracle_lib, page, cap):
    """A prompt step, decode steps and a draft step of four sequences; the window and the pages are those of
    earlier steps; a selection over the same cache."""
    n_seq, m = 4, 300
    c = _cache(n_seq, 120, page, 600, m, cap)
    g = torch.Generator().manual_seed(9)
    qg, lg = (1 + 0.1 * torch.randn(512, generator=g)).cuda(), (1 + 0.1 * torch.randn(512, generator=g)).cuda()
    kv, swa = [np.zeros((0, 288), np.uint8)] * n_seq, [np.zeros((0, 528), np.uint8)] * n_seq
    for k, new in enumerate([[130, 0, 1, 100], [1, 1, 1, 1], [5, 40, 0, 3], [1, 1, 1, 1]]):
        q, lat = _inputs(m, 100 + k)
        c.plan(_i32(new))
        c.write(q, lat, qg, lg)
        out, lse = c.attend()
        scores = torch.rand((m, 608), generator=torch.Generator().manual_seed(k)).cuda()
        sel = torch.empty((m, 64), dtype=torch.int32, device="cuda")
        wsb = lib.csa2_workspace_size(lib.CSA2_OP_TOPK, m, 608, 64)
        tws = torch.empty(max(1, wsb), dtype=torch.uint8, device="cuda")
        lib.csa2_topk(scores, 608, m, c.desc[1], 608, 64, 1, None, sel, tws, wsb)
        out, lse = out.cpu().numpy(), lse.cpu().numpy()
        out_sel, _ = c.attend(sel)
        out_sel, sel = out_sel.cpu().numpy(), sel.cpu().numpy()
        before = c.seq_len.cpu().numpy()
        c.advance()
        assert lib.csa2_get_device_status() == 0
        assert np.array_equal(c.seq_len.cpu().numpy(), before + new)
        t = 0
        got_q = R.bf16_values(_bits(c.q))
        for b, n in enumerate(new):
            if n == 0:
                continue
            pos = before[b] + np.arange(n)
            x = R.norm_rope(lat[t:t + n].float().cpu().numpy(), lg.cpu().numpy(), pos, 1e-6)
            bits = R.round_bf16_bits(x)
            assert np.array_equal(_bits(c.latent[t:t + n]), bits)
            kv[b] = np.concatenate([kv[b], oracle_lib.pack_kv(bits)])
            swa[b] = np.concatenate([swa[b], oracle_lib.pack_swa(bits)])
            want_q = R.norm_rope(q[t:t + n].float().cpu().numpy(), qg.cpu().numpy(), pos[:, None], 1e-6)
            # one rounding to bf16, and fp32 arithmetic: 20 half steps of the row's magnitude are far more than it has
            assert np.abs(got_q[t:t + n] - want_q).max() <= (2.0**-8 + 20 * 2.0**-24) * np.abs(want_q).max()
            for i in {0, n // 2, n - 1}:
                vis = pos[i] + 1
                win = R.swa_values(swa[b][max(0, vis - 128):vis])
                o, le = R.attention(got_q[t + i], np.concatenate([R.kv_values(kv[b][:vis]), win]), pos[i])
                assert row_norm_err(out[t + i], o) <= ATTN_TOL_F32, (k, b, i)
                # fp32 sums of 512 products of bf16 and f16 values: 512 half steps of the sum of their magnitudes
                room = 2.0**-15 * 512**-0.5 * (np.abs(got_q[t + i].astype(np.float64)) @ np.abs(R.kv_values(kv[b][:vis])).T).max()
                assert np.abs(lse[t + i] - le).max() <= room + 1e-6 + 2.0**-23 * np.abs(le).max()
                pick = [j for j in sel[t + i] if j >= 0]
                assert len(pick) == min(64, vis)
                o, _ = R.attention(got_q[t + i], np.concatenate([R.kv_values(kv[b][pick]), win]), pos[i])
                assert row_norm_err(out_sel[t + i], o) <= ATTN_TOL_F32, (k, b, i)
            t += n
        assert np.all(out[t:] == 0) and np.all(np.isneginf(lse[t:]))      # places without a token
    # the cache read back, in sequence order
    for b in range(n_seq):
        n = len(kv[b])
        table = c.table[b].cpu().numpy()
        slots = table[np.arange(n) // page] * page + np.arange(n) % page
        back = c.read(_i32(slots), torch.empty((n, 512), dtype=torch.float32, device="cuda"))
        assert np.array_equal(back.cpu().numpy(), R.kv_values(kv[b]))
    assert lib.csa2_get_device_status() == 0


def _steps(c, news, seeds, m, how):
    outs = []
    for new, seed in zip(news, seeds):
        outs.append(how(_i32(new), *_inputs(m, seed)))
    return outs


def test_a_step_captured_and_replayed(lib):
    """Replays with other inputs in the same places give the bits of eager steps."""
    news, seeds, m = [[30, 200, 1], [1, 1, 1], [1, 0, 2], [1, 1, 1]], [1, 2, 3, 4], 240
    a, b = _cache(3, 60, 16, 400, m, 340), _cache(3, 60, 16, 400, m, 340)
    want = _steps(a, news, seeds, m, lambda n, q, l: [x.clone() for x in a.step(n, q, l)])
    new, q, lat = _i32([0, 0, 0]), *_inputs(m, 99)
    b.step(new, q, lat)                                    # (before capture: the libraries' own set-up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(new, q, lat)
    got = []
    for n, seed in zip(news, seeds):
        x, y = _inputs(m, seed)
        new.copy_(_i32(n)), q.copy_(x), lat.copy_(y)
        graph.replay()
        got.append([z.clone() for z in (b.out, b.lse)])
    torch.cuda.synchronize()
    assert lib.csa2_get_device_status() == 0
    for (o, l), (o2, l2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(l, l2)
    assert torch.equal(a.seq_len, b.seq_len) and torch.equal(a.pages, b.pages) and torch.equal(a.swa, b.swa)


def test_two_at_once_on_other_streams(lib):
    """Two caches stepped on two streams at the same time, neither the current one."""
    m, new = 66, [64, 1, 1]
    def run(streams):
        cs = [_cache(3, 400, 16, 2000, m, 200) for _ in range(2)]
        ins = [[_inputs(m, 10 * s + k) for k in range(6)] for s in range(2)]
        n = _i32(new)
        torch.cuda.synchronize()
        for k in range(6):
            for s in range(2):
                cs[s].step(n, *ins[s][k], stream=streams[s])
        torch.cuda.synchronize()
        return [(c.out.clone(), c.lse.clone(), c.pages.clone(), c.table.clone()) for c in cs]
    cur = torch.cuda.current_stream()
    want = run([cur, cur])
    for _ in range(3):
        got = run([torch.cuda.Stream(), torch.cuda.Stream()])
        for w, g in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w, g))
    assert lib.csa2_get_device_status() == 0


def test_a_cache_that_runs_out_of_pages(lib):
    """The tokens behind the last page write nothing and see what there is; the other sequences go on."""
    c = _cache(2, 3, 16, 100, 40, 160)
    out, lse = c.step(_i32([16, 16]), *_inputs(40, 1))
    assert lib.csa2_get_device_status() == 0
    pages = c.pages.clone()
    out, lse = c.step(_i32([16, 16]), *_inputs(40, 2))     # one page is left
    assert lib.csa2_get_device_status() == BOUNDS
    torch.cuda.synchronize()
    assert (c.table[:, 1] == torch.tensor([2, -1], device="cuda")).all()
    assert torch.equal(c.pages[:2], pages[:2]) and bool((c.desc[5][16:32] == -1).all())
    assert bool(torch.isfinite(out[:32]).all()) and bool((out[32:] == 0).all())


# ------------------------------------------------------------------ attention, the rest of its range
@pytest.mark.parametrize("page", [7, 8, 9])
def test_attn_pages_of_a_few_entries(lib, oracle_lib, page):
    c = Case(oracle_lib, [1000, 129, 8], page, seed=page)
    c.check(lib, _decode_queries([1000, 129, 8]))
    assert lib.csa2_get_device_status() == 0


@pytest.mark.parametrize("n,entries,step", [(256, 600, 32), (160, 512, 16), (100, 2000, 10), (1100, 140, 110)])
def test_attn_runs_of_rows_are_those_rows(lib, oracle_lib, n, entries, step):
    """Many rows at once are dealt to the SMs in other pieces than a few of them."""
    c = Case(oracle_lib, [entries], 64, swa_cap=400, seed=n)
    r = np.random.default_rng(n)
    vis = r.integers(entries // 2, entries + 1, n)
    q = [(0, int(v), int(v) - 1, int(r.integers(0, 400)), 128 if i % 5 else 0) for i, v in enumerate(vis)]
    whole, lse = c.run(lib, q)
    x = c.q
    for i in range(0, n, step):
        part = _attend_rows(lib, c, x[i:i + 3], q[i:i + 3])
        assert row_norm_err(whole[i:i + 3], part[0]) <= 2 * ATTN_TOL_F32, i
        assert np.abs(lse[i:i + 3] - part[1]).max() <= 1e-5
    c.check(lib, q[:2], got=(whole[:2], lse[:2]))
    assert lib.csa2_get_device_status() == 0


def _attend_rows(lib, c, q_bits, queries, params=None, f32=True, sel=None):
    nq, a = len(queries), np.array(queries, np.int64)
    wsb = lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, nq, 0)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    out = torch.empty((nq, 64, 512), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    lse = torch.empty((nq, 64), dtype=torch.float32, device="cuda")
    lib.csa2_paged_attn(_bf16(np.ascontiguousarray(q_bits)), torch.from_numpy(c.pages).cuda(), c.n_pages, c.page, _i32(c.table),
                        c.table.shape[1], len(c.lens), None if sel is None else _i32(sel), 0 if sel is None else sel.shape[1],
                        torch.from_numpy(c.swa).cuda(), c.swa_cap, _i32(a[:, 0]), _i32(a[:, 1]), _i32(a[:, 2]), _i32(a[:, 3]),
                        _i32(a[:, 4]), nq, out, lib.CSA2_OUT_F32 if f32 else lib.CSA2_OUT_BF16, lse, params, ws, wsb)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy()


def test_attn_heads_that_are_not_finite(lib, oracle_lib):
    """An infinity or NaN in a head of a query leaves the other heads, and the other queries, as they are."""
    c = Case(oracle_lib, [700, 40], 64, seed=90)
    q = _decode_queries([700, 40]) + [(0, 650, 649, 0, 128)]
    want, want_l = c.run(lib, q)
    x = c.q.copy()
    x[0, 5, 100], x[0, 63, 511], x[2, 0, 0] = 0x7F80, 0x7FC0, 0xFF80
    out, lse = _attend_rows(lib, c, x, q)
    bad = np.zeros((3, 64), bool)
    bad[0, 5] = bad[0, 63] = bad[2, 0] = True
    assert np.array_equal(out[~bad], want[~bad]) and np.array_equal(lse[~bad], want_l[~bad])
    assert not np.isfinite(out[bad]).all(-1).any()


def test_scale_and_rotation_of_other_parameters(lib, oracle_lib):
    p = lib.default_params()
    p.sm_scale, p.rope_base = 0.03, 500000.0
    c = Case(oracle_lib, [300, 30], 16, seed=91)
    q = _decode_queries([300, 30])
    c.run(lib, q)
    for f32 in (True, False):
        out, lse = _attend_rows(lib, c, c.q, q, p, f32)
        for i, (b, vis, pos, first, cnt) in enumerate(q):
            k = np.concatenate([R.kv_values(R.paged_rows(c.pages, c.table[b], 16, range(vis))),
                                R.swa_values(c.swa[b][(first + np.arange(cnt)) % 128])])
            o, le = R.attention(R.bf16_values(c.q[i]), k, pos, np.float32(0.03), 500000.0)
            assert row_norm_err(out[i], o) <= (ATTN_TOL_F32 if f32 else ATTN_TOL_BF16)
    x = torch.randn((3, 512), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    y = torch.empty_like(x)
    pos = [7, 70_001, 1 << 20]
    lib.csa2_qk_norm_rope(None, 0, None, None, x, 512, None, y, _i32(pos), None, None, 3, 1e-6, None, 0, None, 0, p)
    assert np.array_equal(_bits(y), R.round_bf16_bits(R.norm_rope(x.float().cpu().numpy(), None, pos, 1e-6, 500000.0)))


def test_rows_of_the_same_sequence_and_entry(lib, oracle_lib):
    """The same query twice, and a selection that names an entry more than once: its weight counts as often."""
    c = Case(oracle_lib, [200], 16, seed=92)
    q = [(0, 200, 199, 72, 128), (0, 200, 199, 72, 128)]
    c.run(lib, q)
    x = np.repeat(c.q[:1], 2, 0)
    out, _ = _attend_rows(lib, c, x, q)
    assert np.array_equal(out[0], out[1])
    sel = np.array([[3, 3, 3, 150, 150, -1], [3, 150, 150, 3, 3, 150]])
    out, _ = _attend_rows(lib, c, x, q, sel=sel)
    for i in range(2):
        k = np.concatenate([R.kv_values(R.paged_rows(c.pages, c.table[0], 16, [j for j in sel[i] if j >= 0])),
                            R.swa_values(c.swa[0][(72 + np.arange(128)) % 128])])
        o, _ = R.attention(R.bf16_values(x[i]), k, 199)
        assert row_norm_err(out[i], o) <= ATTN_TOL_F32


def test_offsets_beyond_32_bits(lib, oracle_lib):
    """Records, rows and outputs behind the first 4 GiB of their tensors are those of a small call."""
    page, n_pages = 64, 265_000                            # 16.96 M records, 4.9 GB
    c = Case(oracle_lib, [1000, 70], page, seed=93)
    far = n_pages - c.n_pages
    pages = torch.zeros((n_pages, page, 288), dtype=torch.uint8, device="cuda")
    pages[far:] = torch.from_numpy(c.pages).cuda()
    q = _decode_queries([1000, 70])
    want, want_l = c.run(lib, q)
    table = np.where(c.table >= 0, c.table + far, -1)
    a = np.array(q)
    wsb = lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, 2, 0)
    ws, swa = torch.empty(wsb, dtype=torch.uint8, device="cuda"), torch.from_numpy(c.swa).cuda()
    sel = np.tile(np.arange(0, 70), (2, 1))
    near_sel, _ = _attend_rows(lib, c, c.q, q, sel=sel)
    for s, w in ((None, want), (sel, near_sel)):
        out, lse = torch.empty((2, 64, 512), device="cuda"), torch.empty((2, 64), device="cuda")
        lib.csa2_paged_attn(_bf16(c.q), pages, n_pages, page, _i32(table), table.shape[1], 2, None if s is None else _i32(s),
                            0 if s is None else s.shape[1], swa, 128, _i32(a[:, 0]), _i32(a[:, 1]), _i32(a[:, 2]), _i32(a[:, 3]),
                            _i32(a[:, 4]), 2, out, lib.CSA2_OUT_F32, lse, None, ws, wsb)
        assert np.array_equal(out.cpu().numpy(), w)
    # a cache write there, and records read back into rows behind 4 GiB
    m, slots = 66_000, n_pages * page
    x = torch.randn((64, 64, 512), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    lat = torch.randn((64, 512), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    big = torch.empty((m, 64, 512), dtype=torch.bfloat16, device="cuda")                 # 4.3 GB
    big[-64:] = x
    lats = torch.zeros((m, 512), dtype=torch.bfloat16, device="cuda")
    lats[-64:] = lat
    pos = torch.arange(m, dtype=torch.int32, device="cuda")
    slot = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    slot[-64:] = torch.arange(slots - 64, slots, dtype=torch.int32, device="cuda")
    lib.csa2_qk_norm_rope(big, 32768, None, big, lats, 512, None, lats, pos, slot, None, m, 1e-6, pages, slots, None, 0)
    small_q, small_l = torch.empty_like(x), torch.empty_like(lat)
    small = torch.zeros((64, 288), dtype=torch.uint8, device="cuda")
    lib.csa2_qk_norm_rope(x, 32768, None, small_q, lat, 512, None, small_l, pos[-64:].clone(), _i32(range(64)), None, 64, 1e-6,
                          small, 64, None, 0)
    assert torch.equal(big[-64:], small_q) and torch.equal(lats[-64:], small_l)
    assert torch.equal(pages.view(-1, 288)[-64:], small)
    del big
    n = 2_200_000
    back = torch.empty((n, 512), dtype=torch.float32, device="cuda")                     # 4.5 GB
    where = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    where[-64:] = slot[-64:]
    lib.csa2_cache_read(lib.CSA2_KV_NVFP4, pages, slots, where, n, back, lib.CSA2_OUT_F32)
    assert np.array_equal(back[-64:].cpu().numpy(), R.kv_values(small.cpu().numpy())) and not bool(back[:-64].any())
    assert lib.csa2_get_device_status() == 0
