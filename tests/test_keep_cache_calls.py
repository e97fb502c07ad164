"""PagedCache's bookkeeping of calls that come twice, on the CPU."""
import pytest

torch = pytest.importorskip("torch")

I32 = dict(dtype=torch.int32)


@pytest.fixture
def cache(monkeypatch):
    from compressed_sparse_attention_index_gb300 import decode
    done = []
    for name in ("csa2_page_plan_at", "csa2_attn_weight", "csa2_evict", "csa2_page_trim"):
        monkeypatch.setattr(decode.L, name, lambda *a, _n=name: done.append(_n))
    c = decode.PagedCache(2, 8, 16, 64, 5, device="cpu", voters=5)
    c.done = done
    return c


def test_a_step_is_weighed_once(cache):
    keep = torch.full((2,), 9, **I32)
    for behind in (cache.advance, lambda: cache.accept(torch.ones(2, **I32))):
        cache.plan(torch.zeros(2, **I32), rows=3)
        behind()
        cache.weigh()
        with pytest.raises(ValueError, match="weigh"):
            cache.weigh()
        cache.evict(keep)
        with pytest.raises(ValueError, match="eviction"):
            cache.weigh()
    assert cache.done.count("csa2_attn_weight") == 2


def test_steps_of_a_graph(cache, monkeypatch):
    """The host sees a captured step once, however often it is replayed: weigh behind it is not refused, unless the graph has it."""
    keep, capturing = torch.full((2,), 9, **I32), [True]
    monkeypatch.setattr(cache, "_capturing", lambda: capturing[0])
    cache.plan(torch.zeros(2, **I32), rows=3)
    cache.advance()
    capturing[0] = False
    for _ in range(3):                                    # (a replay each)
        cache.weigh()
        cache.evict(keep)
    cache.plan(torch.zeros(2, **I32), rows=3)             # an eager step again
    cache.advance()
    cache.weigh()
    with pytest.raises(ValueError):
        cache.weigh()
    for last in (cache.weigh, lambda: cache.evict(keep)):
        capturing[0] = True
        cache.plan(torch.zeros(2, **I32), rows=3)
        cache.advance()
        last()
        capturing[0] = False
        with pytest.raises(ValueError):
            cache.weigh()
    capturing[0] = False
    cache.plan(torch.zeros(2, **I32), rows=3)             # weighed once before it is captured on its own
    cache.advance()
    cache.weigh()
    capturing[0] = True
    cache.weigh()
    with pytest.raises(ValueError):
        cache.weigh()


def test_source_refusals(cache):
    cache.plan(torch.zeros(2, **I32), rows=3)
    cache.advance()
    keep = torch.full((2,), 9, **I32)
    for bad in (torch.zeros(2, **I32), torch.zeros((3, 9), **I32), torch.zeros((2, 9)), torch.zeros((9, 2), **I32).t(), torch.zeros((2, 18), **I32)[:, ::2]):
        with pytest.raises(ValueError, match="source"):
            cache.evict(keep, source=bad)
    cache.evict(keep, source=torch.zeros((2, 9), **I32))
    assert cache.done.count("csa2_evict") == 1
