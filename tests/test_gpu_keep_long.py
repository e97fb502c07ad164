"""GPU parity of csa2_attn_weight in runs long enough for a CTA to use every buffer again: stages of records, accumulators, places of
slots, blocks of chunks that take turns at several groups of queries; against 64 bits on the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SMS = 152


def _reference(q, k, lse):
    """(weights, bound) that entries k (fp64 [n][512]) get from one query (fp64 [64][512]), with the bound that
    tests/keep_reference.py derives: fp32 sums of 512 products, cut or rounded, and the exponential."""
    scale = 512 ** -0.5
    w, room = torch.zeros(len(k), dtype=torch.float64, device="cuda"), torch.zeros(len(k), dtype=torch.float64, device="cuda")
    for a in range(0, len(k), 1 << 17):
        x = scale * (k[a:a + (1 << 17)] @ q.T) - lse
        d = 2 * 512 * 2.0**-24 * scale * (k[a:a + (1 << 17)].abs() @ q.abs().T) + 2.0**-20 + 2.0**-22 * lse.abs()
        w[a:a + (1 << 17)] = torch.exp(x).sum(1)
        room[a:a + (1 << 17)] = (torch.exp(x + d) - torch.exp(x)).sum(1)
    return w, room


@pytest.mark.parametrize("lens,counts,page,sel", [
    ([SMS * 20 * 128 + 77], [1], 64, 0),                          # one query: twenty chunks a CTA
    ([SMS * 19 * 128 + 5], [1], 4, 0),                            # records one by one
    ([SMS * 30 * 128 - 1], [3], 48, 0),                           # two groups of up to two, thirty chunks a CTA: two blocks
    ([100, SMS * 10 * 128 + 9, 50, 70, 1], [0, 3, 0, 1, 0], 64, 0),        # more sequences than queries: groups of one, ten chunks a CTA
    ([SMS * 5 * 128 + 300, 40_000], [20, 1], 100, 0),             # more groups than constants have places
    ([5000] * 38, [20] * 38, 64, 512),                            # 760 selections, twenty chunks a CTA
])
def test_weights_of_long_runs(lens, counts, page, sel):
    import compressed_sparse_attention_index_gb300 as lib
    g = torch.Generator(device="cuda").manual_seed(len(lens) + page)
    n_seq, n_q, cols = len(lens), sum(counts), max(-(-n // page) for n in lens)
    have = torch.tensor([-(-n // page) for n in lens], device="cuda")
    n_pages = int(have.sum()) + 2
    ids, col = torch.randperm(n_pages, generator=g, device="cuda"), torch.arange(cols, device="cuda")
    start = torch.cumsum(have, 0) - have
    table = torch.where(col < have[:, None], ids[(start[:, None] + col).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    pages = torch.randint(0, 256, (n_pages * page, 288), generator=g, dtype=torch.uint8, device="cuda")
    pages[:, 256:] = torch.randint(40, 60, (n_pages * page, 32), generator=g, dtype=torch.uint8, device="cuda")
    q = torch.randn((n_q, 64, 512), generator=g, device="cuda").bfloat16()
    first = np.concatenate([[0], np.cumsum(counts)])
    seq = np.repeat(np.arange(n_seq), counts)
    vis = np.array([lens[b] - counts[b] + t + 1 for b in range(n_seq) for t in range(counts[b])])
    lse = torch.tensor(np.log(np.minimum(vis, sel) if sel else vis) + 1.5, device="cuda").float()[:, None] + 0.2 * torch.randn((n_q, 64), generator=g, device="cuda")
    prior = torch.rand(n_pages * page, generator=g, device="cuda")
    picks = None
    if sel:
        picks = torch.stack([torch.randperm(int(v), generator=g, device="cuda")[:sel] for v in vis]).to(torch.int32).contiguous()
    i32 = lambda x: torch.tensor(np.array(x, np.int32), device="cuda")
    out = torch.full((n_pages * page,), -7.0, device="cuda")
    ws = torch.empty(lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, n_q, n_seq, sel), dtype=torch.uint8, device="cuda")
    lib.csa2_attn_weight(q, pages, n_pages, page, table, cols, i32(first), n_seq, picks, sel, i32(vis), lse, n_q, 0.75, prior, out, None, ws, ws.numel())
    again = torch.full_like(out, -7.0)
    lib.csa2_attn_weight(q, pages, n_pages, page, table, cols, i32(first), n_seq, picks, sel, i32(vis), lse, n_q, 0.75, prior, again, None, ws, ws.numel())
    assert lib.csa2_get_device_status() == 0 and torch.equal(out, again)
    want, room = torch.full((n_pages * page,), -7.0, dtype=torch.float64, device="cuda"), torch.zeros(n_pages * page, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if counts[b] == 0:
            continue
        j = torch.arange(n, device="cuda")
        slot = table[b].long()[j // page] * page + j % page
        k = torch.empty((n, 512), device="cuda")
        lib.csa2_cache_read(lib.CSA2_KV_NVFP4, pages, n_pages * page, slot.to(torch.int32), n, k, lib.CSA2_OUT_F32)
        k = k.double()
        got, err = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
        for i in range(first[b], first[b + 1]):
            js = picks[i].long() if sel else torch.arange(int(vis[i]), device="cuda")
            w, e = _reference(q[i].double(), k[js], lse[i].double())
            got.index_add_(0, js, w), err.index_add_(0, js, e)
        want[slot] = 0.75 * prior[slot].double() + got
        room[slot] = err + 2.0**-22 * (0.75 * prior[slot].double() + counts[b] * got)
    assert lib.csa2_get_device_status() == 0
    assert torch.equal(out[room == 0], want[room == 0].float())
    assert bool(((out.double() - want).abs() <= room).all()), float(((out.double() - want).abs() / room.clamp(min=1e-300)).max())
