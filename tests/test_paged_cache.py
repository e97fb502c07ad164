"""PagedCache's own bookkeeping, on the CPU: what a step commits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import paged_reference as R


@pytest.fixture(scope="module")
def cache():
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    return lambda *a, **k: PagedCache(*a, device="cpu", **k)


@pytest.mark.parametrize("n_seq,n_pages,page,max_len,rows,seed", [(3, 20, 16, 100, 40, 0), (5, 9, 4, 60, 16, 1), (2, 30, 1, 50, 25, 2),
                                                                  (1, 6, 7, 40, 8, 3), (9, 12, 8, 64, 64, 4)])
def test_advance_by_what_was_written(cache, n_seq, n_pages, page, max_len, rows, seed):
    """Steps that fit, run out of pages, of rows and of their table's row: lengths, pages and the free list's head."""
    c = cache(n_seq, n_pages, page, max_len, rows)
    r = np.random.default_rng(seed)
    lens, head, table = np.zeros(n_seq, np.int64), 0, np.full(c.table.shape, -1)
    reported = 0
    for _ in range(60):
        new = r.integers(0, 1 + 2 * rows // n_seq, n_seq) * (r.random(n_seq) < 0.6)
        desc, first, totals, planned, fine = R.plan(lens, new, page, n_pages, np.arange(n_pages), head, table, c.swa_cap, rows)
        c.desc.copy_(torch.from_numpy(desc.astype(np.int32)))
        c.first.copy_(torch.from_numpy(first.astype(np.int32))), c.totals.copy_(torch.from_numpy(totals.astype(np.int32)))
        c.advance()
        reported += not fine
        for b in range(n_seq):
            kept = [t for t in range(first[b], min(first[b + 1], rows)) if desc[5][t] >= 0]
            assert kept == list(range(first[b], first[b] + len(kept)))
            before, lens[b] = lens[b], lens[b] + len(kept)
            cols = range(-(-before // page), -(-lens[b] // page))
            for col in cols:
                assert planned[b, col] == head      # the free list names the pages in order
                table[b, col] = head
                head += 1
        assert c.seq_len.tolist() == lens.tolist() and c.free_head.tolist() == [head]
    assert 0 < reported < 60


def test_a_cache_without_a_plan_holds_no_tokens(cache):
    c = cache(3, 8, 1, 64, 5)
    assert c.desc.tolist() == [[0] * 5] * 5 + [[-1] * 5] * 2 and c.first.tolist() == [0] * 4 and c.totals.tolist() == [0, 0]
    c.advance()
    assert c.seq_len.tolist() == [0, 0, 0] and c.free_head.tolist() == [0]


def test_rows_of_a_step(cache):
    """Inputs have as many rows as the step was planned for; the views of a step of r rows are those of a cache of r."""
    c, d = cache(3, 8, 16, 64, 5), cache(3, 8, 16, 64, 2)
    with pytest.raises(ValueError):
        c.plan(torch.zeros(3, dtype=torch.int32), rows=6)
    with pytest.raises(ValueError):
        c.plan(torch.zeros(3, dtype=torch.int32), rows=-1)
    with pytest.raises(ValueError):
        c.step(torch.zeros(3, dtype=torch.int32), torch.zeros((6, 64, 512), dtype=torch.bfloat16), torch.zeros((6, 512), dtype=torch.bfloat16))
    c._use_rows(2)                                        # (as plan does)
    assert c.desc.shape == (7, 2) and c.desc.is_contiguous()
    desc = torch.tensor([[0, 2], [1, 1], [0, 0], [0, 0], [1, 1], [0, 16], [0, 256]], dtype=torch.int32)
    for x in (c, d):
        x.desc.copy_(desc)
        x.advance()
        assert x.seq_len.tolist() == [1, 0, 1] and x.free_head.tolist() == [2]
    with pytest.raises(ValueError):
        c.write(torch.zeros((5, 64, 512), dtype=torch.bfloat16), torch.zeros((5, 512), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        c.attend(torch.zeros((5, 8), dtype=torch.int32))


def test_slots_elsewhere_are_refused(cache):
    """Slots have to lie on the cache's device: the kernel reads them there."""
    c = cache(3, 8, 16, 64, 5)
    with pytest.raises(ValueError):
        c.read(torch.zeros(6, dtype=torch.int32, device="meta"), torch.zeros((6, 512)))
    with pytest.raises(ValueError):
        c.read(torch.zeros(6, dtype=torch.int32), torch.zeros((6, 512), device="meta"))


def test_a_single_row_of_any_stride(cache, monkeypatch):
    """A step of one row: the stride to a next row, which there is not, may be anything."""
    from compressed_sparse_attention_index_gb300 import decode
    seen = []
    monkeypatch.setattr(decode.L, "csa2_qk_norm_rope", lambda *a: seen.append((a[1], a[5])))
    c = cache(1, 8, 16, 64, 1)
    q, lat = torch.zeros((64, 1, 512), dtype=torch.bfloat16).transpose(0, 1), torch.zeros((512, 1), dtype=torch.bfloat16).t()
    assert q.stride(0) == 512 and lat.stride(0) == 1
    c.write(q, lat)
    assert seen == [(64 * 512, 512)]


def test_limits(cache):
    for rows in (0, 65_536):
        with pytest.raises(ValueError):
            cache(3, 8, 16, 64, rows)
    for cap in (-1, 2**30):
        with pytest.raises(ValueError):
            cache(3, 8, 16, 64, 5, swa_cap=cap)


def test_advance_after_a_step_of_other_rows(cache):
    """Descriptors read with other rows than they were planned for name no place outside the state."""
    c = cache(2, 8, 16, 64, 40)
    c._use_rows(4)
    c.desc.copy_(torch.tensor([[0, 0, 1, 1], [1, 2, 60, 61], [0, 1, 59, 60], [0] * 4, [1] * 4, [100, 101, 102, 103], [5] * 4]))
    c._use_rows(40)
    c.advance()                                          # (index_add_ would raise)
    assert c.seq_len.shape == (2,)
