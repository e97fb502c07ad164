"""PagedCache's own bookkeeping of what it keeps, on the CPU: refusals, and the order of its calls."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def cache():
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    return lambda *a, **k: PagedCache(*a, device="cpu", **k)


I32 = dict(dtype=torch.int32)


def test_voters(cache):
    for voters in (-1, 6):
        with pytest.raises(ValueError):
            cache(3, 8, 16, 64, 5, voters=voters)
    c = cache(3, 8, 16, 64, 5)
    assert c.weight is None and c.gone.tolist() == [0] * 3
    for call in (lambda: c.weigh(), lambda: c.evict(torch.zeros(3, **I32))):
        with pytest.raises(ValueError, match="voters"):
            call()
    assert cache(3, 8, 16, 64, 5, voters=4).weight.tolist() == [0.0] * 128


def test_verify_refusals(cache):
    c = cache(2, 8, 16, 64, 5)
    c._use_rows(4)
    tok, p, u, v = torch.zeros(4, **I32), torch.zeros(4, 10), torch.zeros(4), torch.zeros(2)
    bad = [dict(tokens=tok[:3]), dict(tokens=tok.long()), dict(target=p[:3]), dict(target=p.double()), dict(target=p.view(-1)),
           dict(draft=p[:, :9]), dict(draft=p.bfloat16()), dict(u=None), dict(u=u[:3]), dict(v=None), dict(v=u), dict(v=v.double()),
           dict(greedy=True), dict(tokens=torch.zeros(8, **I32)[::2]), dict(u=torch.zeros(8)[::2]),
           dict(target=torch.zeros(10, 4).t(), draft=None)]
    for kw in bad:
        with pytest.raises(ValueError):
            c.verify(**{**dict(tokens=tok, target=p, draft=p, u=u, v=v), **kw})


def test_order_of_calls(cache, monkeypatch):
    from compressed_sparse_attention_index_gb300 import decode
    done = []
    for name in ("csa2_page_plan_at", "csa2_attn_weight", "csa2_evict", "csa2_page_trim", "csa2_paged_attn"):
        monkeypatch.setattr(decode.L, name, lambda *a, _n=name: done.append(_n))
    c = cache(2, 8, 16, 64, 5, voters=3)
    keep = torch.full((2,), 9, **I32)
    with pytest.raises(ValueError):
        c.weigh()                                         # nothing to weigh yet
    c.plan(torch.zeros(2, **I32), rows=3)
    for call in (c.weigh, lambda: c.evict(keep)):
        with pytest.raises(ValueError, match="advance"):
            call()
    c.advance()
    c.weigh()
    c.evict(keep)
    with pytest.raises(ValueError, match="eviction"):
        c.weigh()                                         # the entries have moved
    c.evict(keep)
    c.plan(torch.zeros(2, **I32), rows=5)
    c.advance()
    with pytest.raises(ValueError, match="3 rows"):
        c.weigh()
    for bad in (keep[:1], keep.long(), torch.zeros(4, **I32)[::2]):
        with pytest.raises(ValueError):
            c.evict(bad)
        with pytest.raises(ValueError):
            c.accept(bad)
    with pytest.raises(ValueError):
        c._use_rows(2)
        c.weigh(sel=torch.zeros((3, 8), **I32))
    assert done.count("csa2_attn_weight") == 1 and done.count("csa2_evict") == 2


def test_accept_bookkeeping(cache, monkeypatch):
    """Lengths, pages and what the queries see, with the trim's own restatement in its place."""
    from compressed_sparse_attention_index_gb300 import decode
    from tests import keep_reference as K
    c = cache(3, 12, 4, 40, 9)

    def trim(length, to, n_seq, page, n_pages, free, n_free, head, table, stride, stream=None):
        f, h, t, fine = K.trim(length.tolist(), to.tolist(), page, n_pages, free.numpy(), int(head[0]), table.numpy())
        assert fine
        free.copy_(torch.from_numpy(f)), head.fill_(int(h)), table.copy_(torch.from_numpy(t))
    monkeypatch.setattr(decode.L, "csa2_page_trim", trim)
    # 4, 3 and 2 tokens of empty sequences on pages 0, 1, 2: the first keeps two, the second none, the third more than it has
    c._use_rows(9)
    c.desc.copy_(torch.tensor([[0] * 4 + [1] * 3 + [2] * 2, [1, 2, 3, 4, 1, 2, 3, 1, 2], [0, 1, 2, 3, 0, 1, 2, 0, 1], [0] * 9, [1] * 9,
                               [0, 1, 2, 3, 4, 5, 6, 8, 9], [-1] * 9]))
    c.first.copy_(torch.tensor([0, 4, 7, 9]))
    c.table[0, 0], c.table[1, 0], c.table[2, 0] = 0, 1, 2
    c.accept(torch.tensor([2, -3, 7], **I32))
    assert c.seq_len.tolist() == [2, 0, 2] and c.free_head.tolist() == [2]
    assert c.table[:, 0].tolist() == [0, -1, 2] and c.free[2].item() == 1
    assert c._d[1].tolist() == [1, 2, 0, 0, 0, 0, 0, 1, 2]
