"""PagedCache over several steps against a plain restatement that keeps every
sequence's records: steps that fit, and steps of which a part does not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import paged_reference as R  # noqa: E402
from parity import ATTN_TOL_F32, row_norm_err  # noqa: E402
from test_gpu_paged import BOUNDS, _bits, _i32  # noqa: E402
from test_gpu_paged_run import _inputs  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


class Sequences:
    """A PagedCache (fp32 outputs) and what its sequences hold, record by record."""

    def __init__(self, oracle_lib, n_seq, n_pages, page, max_len, max_tokens, cap=None):
        import compressed_sparse_attention_index_gb300 as lib
        from compressed_sparse_attention_index_gb300.decode import PagedCache
        kw = {} if cap is None else {"swa_cap": cap}
        self.c = PagedCache(n_seq, n_pages, page, max_len, max_tokens, out_dtype=lib.CSA2_OUT_F32, **kw)
        self.lib, self.oracle, self.n_seq, self.page = lib, oracle_lib, n_seq, page
        self.kv = [np.zeros((0, 288), np.uint8)] * n_seq
        self.swa = [np.zeros((0, 528), np.uint8)] * n_seq
        self.seed = 0

    def step(self, new, kept=None, first=None, status=0, rows=None, every=1):
        """A step of `new` tokens a sequence, of which kept[b] are written (the others in
        status); first[b]: where sequence b's tokens begin in the step."""
        kept = new if kept is None else kept
        first = np.cumsum([0] + list(new))[:-1] if first is None else first
        c, cap = self.c, self.c.swa_cap
        self.seed += 1
        q, lat = _inputs(c.max_tokens if rows is None else rows, self.seed)
        out, lse = (x.cpu().numpy() for x in c.step(_i32(new), q, lat))
        assert self.lib.csa2_get_device_status() == status
        got_q, w = R.bf16_values(_bits(c.q)), min(128, cap)
        dead = np.ones(len(out), bool)
        for b, n in enumerate(kept):
            held, t = len(self.kv[b]), first[b]
            dead[t:t + new[b]] = False
            if n == 0:
                continue
            bits = R.round_bf16_bits(R.norm_rope(lat[t:t + n].float().cpu().numpy(), None, held + np.arange(n), 1e-6))
            self.kv[b] = np.concatenate([self.kv[b], self.oracle.pack_kv(bits)])
            self.swa[b] = np.concatenate([self.swa[b], self.oracle.pack_swa(bits)])
            for i in sorted({0, 1, n - 1, *range(0, n, every)}):
                if i >= n:
                    continue
                vis = held + i + 1
                k = np.concatenate([R.kv_values(self.kv[b][:vis]), R.swa_values(self.swa[b][max(0, vis - w):vis])])
                o, le = R.attention(got_q[t + i], k, vis - 1)
                assert row_norm_err(out[t + i], o) <= ATTN_TOL_F32, (b, i)
                # fp32 sums of 512 products: 512 half steps of the sum of their magnitudes
                room = 2.0**-15 * 512**-0.5 * (np.abs(got_q[t + i].astype(np.float64)) @ np.abs(k).T).max()
                assert np.abs(lse[t + i] - le).max() <= room + 1e-6 + 2.0**-23 * np.abs(le).max()
        assert np.all(out[dead] == 0) and np.all(np.isneginf(lse[dead]))
        self.check_state()

    def check_state(self):
        """The lengths, the pages and the records of the main cache are the model's."""
        n = [len(x) for x in self.kv]
        cols = [-(-x // self.page) for x in n]
        assert self.c.seq_len.tolist() == n and self.c.free_head.tolist() == [sum(cols)]
        table = self.c.table.cpu().numpy()
        ids = [int(i) for b in range(self.n_seq) for i in table[b, :cols[b]]]
        assert len(set(ids)) == len(ids) and all(0 <= i < self.c.n_pages for i in ids)
        pages = self.c.pages.cpu().numpy()
        for b in range(self.n_seq):
            j = np.arange(n[b])
            assert np.array_equal(pages[table[b, j // self.page], j % self.page], self.kv[b])


# ------------------------------------------------------------------ the window's ring
def test_prompts_and_drafts_through_the_default_ring(lib, oracle_lib):
    """Every token of a step sees its own window: prompts longer than a window, drafts behind a full one."""
    s = Sequences(oracle_lib, 3, 60, 16, 500, 210)
    for new in ([200, 1, 0], [2, 5, 3], [1, 1, 1], [64, 0, 140], [2, 2, 2]):
        s.step(new)


@pytest.mark.parametrize("cap", [128, 150, 64, 1])
def test_a_ring_too_short_for_a_sequences_tokens(lib, oracle_lib, cap):
    """A sequence whose step would overwrite its own windows gets no tokens and is reported; the others go on."""
    w, s = min(128, cap), Sequences(oracle_lib, 3, 60, 16, 500, 3 * cap + 5, cap)
    s.step([cap + 1, cap, 1], [0, cap, 1], [0, 0, cap], BOUNDS)      # (from nothing, a ring of tokens is well)
    s.step([1, 1, 1])
    many = cap + 1 - w                                                # what a full window leaves room for
    s.step([many, many, many])
    if cap > 1:
        s.step([0, many + 1, 1], [0, 0, 1], [0, 0, 0], BOUNDS)
        s.step([2**31 - 1, 0, 0], [0, 0, 0], [0, 0, 0], BOUNDS)
    s.step([1, 1, 1])


def test_a_cache_without_a_window(lib, oracle_lib):
    s = Sequences(oracle_lib, 2, 60, 16, 500, 210, 0)
    s.step([200, 3])
    s.step([1, 40])


def test_tokens_without_a_descriptor_take_no_ring_slot(lib):
    """A token keeps its window record where only dropped tokens would have taken its slot."""
    cap, rows = 32, 20
    desc = torch.full((7, rows), -77, dtype=torch.int32, device="cuda")
    first, totals = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    table = _i32(np.arange(60).reshape(2, 30))
    lib.csa2_page_plan(_i32([10, 300]), _i32([5, 60]), 2, 16, 64, _i32(range(60, 64)), 4, None, table, 30, cap, desc, rows, first, totals)
    assert lib.csa2_get_device_status() == BOUNDS
    pos = np.concatenate([np.arange(10, 15), np.arange(300, 315)])
    assert desc[2].tolist() == pos.tolist() and first.tolist() == [0, 5, 65]
    assert desc[6].tolist() == [(0 if i < 5 else cap) + p % cap for i, p in enumerate(pos)]
    # 40 rows: tokens 300 .. 334, of which 300 .. 302 give way to 332 .. 334
    desc = torch.full((7, 40), -77, dtype=torch.int32, device="cuda")
    lib.csa2_page_plan(_i32([10, 300]), _i32([5, 60]), 2, 16, 64, _i32(range(60, 64)), 4, None, table, 30, cap, desc, 40, first, totals)
    assert lib.csa2_get_device_status() == BOUNDS
    assert desc[6][5:].tolist() == [-1] * 3 + [cap + p % cap for p in range(303, 335)]


# ------------------------------------------------------------------ what a step commits
@pytest.mark.parametrize("page", [16, 1, 7])
def test_steps_beyond_the_last_page(lib, oracle_lib, page):
    """Tokens without a page are reported and not part of their sequences; what comes after sees the others alone."""
    n_pages = -(-10 // page) + -(-16 // page) + -(-22 // page) - -(-10 // page)
    s = Sequences(oracle_lib, 2, n_pages, page, 100, 40)
    s.step([10, 16])
    s.step([12, 9], [12, -(-16 // page) * page - 16], status=BOUNDS)
    room = -(-22 // page) * page - 22
    s.step([min(room, 3), 0])
    s.step([0, 9], [0, 0], status=BOUNDS)
    s.step([0, 0])


def test_steps_of_more_tokens_than_rows(lib, oracle_lib):
    s = Sequences(oracle_lib, 3, 60, 16, 300, 40)
    s.step([30, 200, 1], [30, 10, 0], status=BOUNDS)
    s.step([1, 1, 1])
    s.step([0, 41, 5], [0, 40, 0], status=BOUNDS)
    s.step([20, 10, 10])


def test_a_sequence_beyond_its_row_of_the_table(lib, oracle_lib):
    s = Sequences(oracle_lib, 2, 60, 16, 32, 40)
    s.step([30, 5])
    s.step([3, 5], [0, 5], [0, 0], BOUNDS)
    s.step([2, 5])
    s.step([1, 5], [0, 5], [0, 0], BOUNDS)


# ------------------------------------------------------------------ streams
def test_a_new_cache_is_whole_on_every_stream(lib):
    """The constructor's fills, behind whatever its stream holds, are over when it returns."""
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    new, ins = _i32([3, 1]), _inputs(8, 1)
    want = [x.clone() for x in PagedCache(2, 30, 16, 200, 8).step(new, *ins)]
    torch.cuda.synchronize()
    for _ in range(10):
        a @ a
    c = PagedCache(2, 200_000, 16, 200, 8)                            # 0.9 GB of pages
    assert torch.cuda.current_stream().query()
    s = torch.cuda.Stream()
    got = c.step(new, *ins, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got)) and lib.csa2_get_device_status() == 0


# ------------------------------------------------------------------ rows
def test_a_step_works_on_the_rows_it_is_given(lib, oracle_lib):
    """A cache for long prompts steps a few tokens on a few rows: the bits of a small cache, the rows behind untouched."""
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    big, small = PagedCache(4, 60, 16, 300, 512, 640), PagedCache(4, 60, 16, 300, 8, 640)
    for k, new in enumerate([[2, 1, 4, 1], [1, 1, 1, 1], [0, 3, 0, 0]]):
        for x in (big.out, big.lse, big.q, big.latent):
            x.fill_(7.0)
        q, lat = _inputs(8, k)
        got, want = big.step(_i32(new), q, lat), small.step(_i32(new), q, lat)
        for x, y in zip(got, want):
            assert x.shape == y.shape and torch.equal(x, y)
        assert torch.equal(big.desc, small.desc) and torch.equal(big.first, small.first)
        for x in (big.out, big.lse, big.q, big.latent):
            assert bool((x[8:] == 7.0).all())
    # a step of another number of rows, a captured one, a longer one again
    s = Sequences(oracle_lib, 3, 60, 16, 300, 200)
    s.step([40, 1, 100], rows=150)
    s.step([1, 1, 1], rows=3)
    s.step([5, 0, 60])
    s.step([1, 3, 1], [1, 2, 0], status=BOUNDS, rows=3)
    assert torch.equal(big.seq_len, small.seq_len) and torch.equal(big.pages, small.pages)


def test_a_step_of_a_few_rows_captured(lib):
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    a, b = PagedCache(3, 60, 16, 300, 64), PagedCache(3, 60, 16, 300, 64)
    x, y = _inputs(64, 5)
    for c in (a, b):
        c.step(_i32([40, 3, 20]), x, y)
    new, q, lat = _i32([0, 0, 0]), *_inputs(3, 6)
    b.step(new, q, lat)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(new, q, lat)
    for k in range(3):
        n, (u, v) = _i32([1, k % 2, 1]), _inputs(3, 10 + k)
        want = a.step(n, u, v)
        new.copy_(n), q.copy_(u), lat.copy_(v)
        graph.replay()
        assert torch.equal(want[0], b.out[:3]) and torch.equal(want[1], b.lse[:3])
    torch.cuda.synchronize()
    assert torch.equal(a.seq_len, b.seq_len) and torch.equal(a.pages, b.pages) and lib.csa2_get_device_status() == 0


def test_another_current_device(lib, monkeypatch):
    """The kernels would read the cache of this device from that one."""
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    c, new, ins = PagedCache(2, 30, 16, 200, 8), _i32([3, 1]), _inputs(8, 1)
    want = [x.clone() for x in c.step(new, *ins)]
    here = torch.cuda.current_device()
    slots, out = _i32([0]), torch.empty((1, 512), device="cuda")
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: here + 1)
        for call in (lambda: c.plan(new), lambda: c.write(*ins), c.attend, lambda: c.read(slots, out), lambda: c.step(new, *ins)):
            with pytest.raises(ValueError):
                call()
    assert torch.equal(c.attend()[0], want[0])
