"""A run of the operators that decide what a paged cache keeps, together, through PagedCache: steps of drafts that are
verified and accepted in part, weighed, and now and then cut down, against a model of the cache in plain Python."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import keep_reference as K  # noqa: E402
from tests import paged_reference as R  # noqa: E402

V = 500


def _i32(x):
    return torch.from_numpy(np.array(x, np.int32)).cuda()


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Model:
    """The sequences' entries (latents), all their positions' latents (the windows), and what the cache says of them."""

    def __init__(self, n_seq):
        self.entries, self.past, self.gone = [[] for _ in range(n_seq)], [[] for _ in range(n_seq)], [0] * n_seq


def _slots(c, b, n):
    table = c.table[b].cpu().numpy()
    j = np.arange(n)
    return table[j // c.page_size] * c.page_size + j % c.page_size


def _check_pages(c):
    """Every page is on one column or free, once; the columns are those of the lengths."""
    table, head = c.table.cpu().numpy(), int(c.free_head.item())
    used = []
    for b, n in enumerate(c.seq_len.tolist()):
        cols = -(-n // c.page_size)
        used += table[b, :cols].tolist()
        assert np.all(table[b, :cols] >= 0)
    assert sorted(used + c.free[head:].tolist()) == list(range(c.n_pages)) and head == len(used)


def _probabilities(r, n):
    x = 2 * r.normal(size=(n, V))
    e = lambda y: np.exp(y) / np.exp(y).sum(1, keepdims=True)
    return e(x), e(x + 0.4 * r.normal(size=(n, V)))


@pytest.mark.parametrize("page,seed", [(16, 0), (7, 1), (64, 2)])
def test_run(oracle_lib, page, seed):
    import compressed_sparse_attention_index_gb300 as lib
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    r, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    n_seq, most = 3, 160
    c = PagedCache(n_seq, 3 * 420 // page, page, 600, most, out_dtype=lib.CSA2_OUT_F32, voters=40)
    m = Model(n_seq)
    for step in range(10):
        prompt = step == 0
        new = [150, 1, 9] if prompt else [int(x) for x in r.integers(1, 7, n_seq)]
        if step == 4:
            new[1] = 0
        rows = sum(new) + (3 if step % 3 == 2 else 0)                 # (some rows without a token)
        q = torch.randn((rows, 64, 512), generator=g).bfloat16().cuda()
        c.plan(_i32(new), rows=rows)
        c.write(q, (2 * torch.randn((rows, 512), generator=g)).bfloat16().cuda())
        out, lse = c.attend()
        lat, qn = _bits(c.latent[:rows]), _bits(c.q[:rows])
        # ------------------------------------------------ attention over places, windows of positions
        for b in range(n_seq):
            first = sum(new[:b])
            for t in {0, new[b] - 1} if new[b] else ():
                i = first + t
                entries = m.entries[b] + list(lat[first:i + 1])
                past = (m.past[b] + list(lat[first:i + 1]))[-128:]
                pos = m.gone[b] + len(entries) - 1
                o, le = oracle_lib.sparse_attn_lse(qn[i], oracle_lib.pack_kv(np.array(entries)), oracle_lib.pack_swa(np.array(past)), pos)
                got = out[i].cpu().numpy()
                assert np.abs(got - o).max(1).max() <= 2e-3 * np.abs(o).max() and np.allclose(lse[i].cpu().numpy(), le, atol=1e-4)
        # ------------------------------------------------ which tokens stay
        if prompt:
            kept = new
            c.advance()
        else:
            target, draft = _probabilities(r, rows)
            tok = r.integers(0, V, rows)
            for i in range(rows - 1):
                tok[i + 1] = min(V - 1, np.searchsorted(np.cumsum(draft[i]), r.random()))
            u, v = r.random(rows).astype(np.float32), r.random(n_seq).astype(np.float32)
            first = np.concatenate([[0], np.cumsum(new)])
            P, D = torch.from_numpy(target).float().cuda(), torch.from_numpy(draft).float().cuda()
            got = c.verify(_i32(tok), P, D, torch.from_numpy(u).cuda(), torch.from_numpy(v).cuda())
            want = K.verify(False, P.double().cpu().numpy(), D.double().cpu().numpy(), V, tok, first, u, v)
            assert got[0].tolist() == want[0].tolist() and got[1].tolist() == want[1].tolist()
            kept = want[0].tolist()
            c.accept()
        before = c.weight.cpu().numpy().copy()
        for b in range(n_seq):
            first = sum(new[:b])
            m.entries[b] += list(lat[first:first + kept[b]])
            m.past[b] += list(lat[first:first + kept[b]])
        assert c.seq_len.tolist() == [len(e) for e in m.entries] and c.gone.tolist() == m.gone
        _check_pages(c)
        # ------------------------------------------------ their weights
        if rows > 40:
            with pytest.raises(ValueError):
                c.weigh()
        else:
            c.weigh(decay=0.9)
            first = np.concatenate([[0], np.cumsum(new)])
            n_vis = np.zeros(rows, np.int64)
            for b in range(n_seq):
                n_vis[first[b]:first[b] + kept[b]] = len(m.entries[b]) - kept[b] + 1 + np.arange(kept[b])
            want, room, fine = K.attn_weight(R.bf16_values(qn).astype(np.float64), c.pages.cpu().numpy(), page, c.table.cpu().numpy(), first,
                                             None, n_vis, lse.cpu().numpy(), 0.9, before, before)
            assert fine and np.all(np.abs(c.weight.cpu().numpy() - want) <= room)
        # (an entry's weight is nowhere else: places without an entry weigh nothing)
        w = c.weight.cpu().numpy()
        held = np.concatenate([_slots(c, b, len(m.entries[b])) for b in range(n_seq)]).astype(np.int64)
        assert np.count_nonzero(np.delete(w, held)) == 0
        # ------------------------------------------------ and which entries
        if step in (3, 5, 6, 8):
            keep, recent = ([60, 200, 5], 4) if step != 6 else ([0, 3, 30], 50)
            for b in range(n_seq):
                n, k = len(m.entries[b]), min(keep[b], len(m.entries[b]))
                x, last = w[_slots(c, b, n)], min(recent, k)
                order = sorted(range(n - last), key=lambda j: (-x[j], j))[:k - last]
                m.entries[b] = [m.entries[b][j] for j in sorted(order) + list(range(n - last, n))]
                m.gone[b] += n - k
            c.evict(_i32(keep), recent)
            _check_pages(c)
            with pytest.raises(ValueError):
                c.weigh()
        assert c.seq_len.tolist() == [len(e) for e in m.entries] and c.gone.tolist() == m.gone
        for b in range(n_seq):
            n = len(m.entries[b])
            if n:
                rec = c.pages.view(-1, 288)[_i32(_slots(c, b, n)).long()].cpu().numpy()
                assert np.array_equal(rec, oracle_lib.pack_kv(np.array(m.entries[b])))
        assert lib.csa2_get_device_status() == 0


def _step_inputs(seed, rows):
    g = torch.Generator().manual_seed(seed)
    p = torch.softmax(2 * torch.randn((rows, V), generator=g), 1)
    return dict(q=torch.randn((rows, 64, 512), generator=g).bfloat16().cuda(), latent=torch.randn((rows, 512), generator=g).bfloat16().cuda(),
                target=p.cuda(), draft=torch.softmax(torch.log(p) + 0.4 * torch.randn((rows, V), generator=g), 1).cuda(),
                tokens=torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).cuda(), u=(0.2 * torch.rand(rows, generator=g)).cuda(),
                v=torch.rand(2, generator=g).cuda())


def _drafted(c, x, new, keep, evict):
    c.plan(new, rows=x["q"].shape[0])
    c.write(x["q"], x["latent"])
    c.attend()
    c.verify(x["tokens"], x["target"], x["draft"], x["u"], x["v"])
    c.accept()
    c.weigh(decay=0.5)
    if evict:
        c.evict(keep, 20)


def _state(c):
    return {k: getattr(c, k).clone() for k in ("pages", "swa", "table", "seq_len", "free_head", "free", "gone", "weight", "kept", "next")}


def test_captured_and_replayed():
    """A captured step, its eviction included, replayed with other inputs: the eager one's state, bit for bit; and on a
    stream of its own, beside another cache's steps."""
    import compressed_sparse_attention_index_gb300 as lib
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    new, keep = _i32([4, 3]), _i32([90, 1000])
    make = lambda: PagedCache(2, 60, 16, 400, 100, voters=8)
    eager, graph, other = make(), make(), make()
    for c in (eager, graph, other):
        c.step(_i32([60, 37]), **{k: v for k, v in _step_inputs(1, 97).items() if k in ("q", "latent")})
    x = _step_inputs(2, 7)
    before = _state(graph)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                         # (its kernels are loaded before the capture)
        _drafted(other, x, new, keep, True)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _drafted(graph, x, new, keep, True)
    for k, v in before.items():
        assert torch.equal(getattr(graph, k), v), k       # nothing ran yet
    for seed in (2, 3, 4, 5, 6, 7, 8, 9):
        y = _step_inputs(seed, 7)
        for k in x:
            x[k].copy_(y[k])
        g.replay()
        with torch.cuda.stream(side):
            _drafted(other, _step_inputs(seed + 50, 7), new, keep, seed % 2 == 0)
        _drafted(eager, y, new, keep, True)
        torch.cuda.synchronize()
        a, b = _state(eager), _state(graph)
        for k in a:
            assert torch.equal(a[k].view(torch.uint8) if a[k].dtype == torch.float32 else a[k], b[k].view(torch.uint8) if b[k].dtype == torch.float32 else b[k]), (seed, k)
    assert eager.seq_len[0] == 90 and eager.gone[0] > 0
    _check_pages(eager), _check_pages(other)
    assert lib.csa2_get_device_status() == 0


def test_same_bits_on_every_call(oracle_lib):
    """Weights of drafts, dense and selected, over entries that several queries share."""
    import compressed_sparse_attention_index_gb300 as lib
    from tests.test_gpu_keep import _weigh, _weigh_case
    for sel in (0, 60):
        c = _weigh_case(oracle_lib, 3, [700, 400, 90], 16, [5, 6, 4], sel)
        first = _weigh(lib, c)
        for _ in range(20):
            assert torch.equal(_weigh(lib, c).view(torch.int32), first.view(torch.int32))


def test_on_another_stream(oracle_lib):
    import compressed_sparse_attention_index_gb300 as lib
    from tests.test_gpu_keep import _weigh, _weigh_case
    c = _weigh_case(oracle_lib, 6, [900, 300], 64, [3, 1])
    want = _weigh(lib, c)
    s = torch.cuda.Stream()
    out = torch.full_like(want, -7.0)
    torch.cuda.synchronize()
    _weigh(lib, c, stream=s, out=out)
    s.synchronize()
    assert torch.equal(out, want)


_FIRST_CALLS = """
import torch
import compressed_sparse_attention_index_gb300 as lib
n, page = 70_000, 16
cols = n // page + 1
i32 = dict(dtype=torch.int32, device="cuda")
pages = torch.randint(0, 256, (cols, page, 288), dtype=torch.uint8, device="cuda")
weight = torch.rand(cols * page, device="cuda")
was, old = pages.view(-1, 288).clone(), weight.clone()
table, lens, keep = torch.arange(cols, **i32), torch.tensor([n], **i32), torch.tensor([n // 2], **i32)
p, u, v = torch.softmax(torch.randn(2, 5000, device="cuda"), 1), torch.tensor([0.5, 0.5], device="cuda"), torch.tensor([0.25], device="cuda")
tokens, first, kept, after = torch.tensor([1, 2], **i32), torch.tensor([0, 2], **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
from_ = torch.full((1, n), -1, **i32)
ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_EVICT, 1, cols * page), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    lib.csa2_evict(pages, weight, cols, page, table, cols, lens, keep, 1, 10, pages, weight, cols, table, cols, lens, from_, n, ws, ws.numel())
    lib.csa2_verify_drafts(lib.CSA2_VERIFY_SAMPLE, p, 5000, None, 0, lib.CSA2_PROB_F32, 5000, tokens, first, 1, 2, u, v, kept, after)
assert lens.item() == n
g.replay()
torch.cuda.synchronize()
assert lib.csa2_get_device_status() == 0 and lens.item() == n // 2
j = from_[0, :n // 2].long()
assert torch.equal(pages.view(-1, 288)[:n // 2], was[j]) and torch.equal(weight[:n // 2], old[j])
heaviest = torch.topk(old[:n - 10], n // 2 - 10).values
assert torch.equal(torch.sort(old[j[:-10]], descending=True).values, heaviest) and torch.equal(j[-10:], torch.arange(n - 10, n, device="cuda"))
assert kept.item() == (2 if 0.5 < p[0, 2].item() else 1) and after.item() >= 0
print("first calls captured")
"""


def test_first_calls_of_a_process_captured():
    """What is set up once a device is set up in a capture too."""
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "first calls captured" in r.stdout, r.stdout + r.stderr
