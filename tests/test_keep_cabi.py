"""The entry points that decide what a paged cache keeps reject bad arguments on the host, before anything
is launched (no GPU here), and their plain restatements hold."""
import numpy as np
import pytest

from tests import keep_reference as K
from tests import paged_reference as R

INVALID, UNSUP, WS = 1, 2, 6
FAKE = 1 << 20                                     # never dereferenced: rejected first
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


def _weigh(L, **kw):
    a = dict(q=FAKE, pages=FAKE, n_pages=100, page=64, table=FAKE, stride=8, first=FAKE, n_seq=2, sel=None, sel_stride=0,
             n_vis=FAKE, lse=FAKE, n_q=2, decay=1.0, prior=None, weight=FAKE, params=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return L.csa2_attn_weight(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_q=-1), INVALID), (dict(n_seq=-1), INVALID), (dict(n_pages=0), INVALID), (dict(page=0), INVALID),
    (dict(stride=0), INVALID), (dict(decay=NAN), INVALID), (dict(decay=INF), INVALID), (dict(sel=FAKE, sel_stride=0), INVALID),
    (dict(sel=FAKE, sel_stride=513), INVALID), (dict(n_q=65536), UNSUP), (dict(n_seq=16385), UNSUP),
    (dict(stride=1 << 31), UNSUP), (dict(n_pages=1 << 26), UNSUP), (dict(stride=1 << 26), UNSUP),
    (dict(page=1, stride=2**31 - 255, n_q=1), UNSUP), (dict(page=1, stride=2**31 - 256, n_q=1, q=None), INVALID), (dict(n_q=60000, stride=1 << 20), UNSUP), (dict(q=FAKE + 8), INVALID), (dict(pages=FAKE + 16), INVALID),
    (dict(table=None), INVALID), (dict(first=None), INVALID), (dict(n_vis=None), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(prior=FAKE + 1), INVALID), (dict(weight=None), INVALID), (dict(ws=None), WS), (dict(ws=FAKE + 128), WS),
    (dict(ws_bytes=0), WS), (dict(n_q=0, q=None), 0), (dict(n_seq=0, first=None), 0)])
def test_weight_refusals(lib, kw, code):
    assert _weigh(lib.load(), **kw) == code


def _evict(L, **kw):
    a = dict(pages=FAKE, weight=FAKE, n_pages=100, page=64, table=FAKE, stride=8, seq_len=FAKE, keep=FAKE, n_seq=2,
             recent=4, dst=2 * FAKE, dst_weight=2 * FAKE, n_dst=50, dst_table=2 * FAKE, dst_stride=4, new_len=FAKE,
             from_=None, from_stride=0, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return L.csa2_evict(*a.values(), None)


HERE = dict(dst=FAKE, dst_weight=FAKE, n_dst=100, dst_table=FAKE, dst_stride=8)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), INVALID), (dict(n_pages=0), INVALID), (dict(page=0), INVALID), (dict(stride=0), INVALID),
    (dict(recent=-1), INVALID), (dict(n_dst=0), INVALID), (dict(dst_stride=0), INVALID), (dict(from_=FAKE), INVALID),
    (dict(n_seq=16385), UNSUP), (dict(stride=1 << 26), UNSUP), (dict(dst_stride=1 << 26), UNSUP),
    (dict(page=1, stride=2**31 - 255), UNSUP), (dict(page=1, dst_stride=2**31 - 255), UNSUP),
    (dict(n_pages=1 << 26), UNSUP), (dict(n_dst=1 << 26), UNSUP), (dict(pages=FAKE + 16), INVALID),
    (dict(dst=FAKE + 16), INVALID), (dict(weight=FAKE + 4), INVALID), (dict(dst_weight=FAKE + 2), INVALID),
    (dict(table=None), INVALID), (dict(dst_table=None), INVALID), (dict(seq_len=None), INVALID), (dict(keep=None), INVALID),
    (dict(new_len=None), INVALID), (dict(from_=FAKE + 2, from_stride=4), INVALID),
    # in place means all of the source
    (dict(HERE, dst_weight=2 * FAKE), INVALID), (dict(HERE, n_dst=99), INVALID), (dict(HERE, dst_stride=7), INVALID),
    (dict(HERE, ws=None), WS), (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(ws_bytes=1000), WS),
    (dict(n_seq=0, seq_len=None), 0)])
def test_evict_refusals(lib, kw, code):
    assert _evict(lib.load(), **kw) == code


def _trim(L, **kw):
    a = dict(length=FAKE, new_len=FAKE, n_seq=2, page=64, n_pages=100, free=FAKE, n_free=100, head=FAKE, table=FAKE, stride=8)
    a.update(kw)
    return L.csa2_page_trim(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), INVALID), (dict(page=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_free=-1), INVALID),
    (dict(stride=0), INVALID), (dict(n_seq=16385), UNSUP), (dict(stride=1 << 31), UNSUP), (dict(n_pages=1 << 26), UNSUP),
    (dict(length=None), INVALID), (dict(new_len=FAKE + 2), INVALID), (dict(free=None), INVALID), (dict(head=None), INVALID),
    (dict(table=None), INVALID), (dict(n_seq=0, length=None), 0)])
def test_trim_refusals(lib, kw, code):
    assert _trim(lib.load(), **kw) == code


def _verify(L, **kw):
    a = dict(mode=0, target=FAKE, t_stride=1000, draft=FAKE, d_stride=1000, dtype=1, vocab=1000, tokens=FAKE, first=FAKE,
             n_seq=2, n_rows=6, u=FAKE, v=FAKE, kept=FAKE, next=FAKE, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return L.csa2_verify_drafts(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(mode=2), INVALID), (dict(dtype=3), INVALID), (dict(n_seq=-1), INVALID), (dict(n_rows=-1), INVALID),
    (dict(vocab=0), INVALID), (dict(t_stride=999), INVALID), (dict(d_stride=999), INVALID), (dict(mode=1), INVALID),
    (dict(n_seq=16385), UNSUP), (dict(n_rows=65536), UNSUP), (dict(vocab=(1 << 28) + 1, t_stride=1 << 29, d_stride=1 << 29), UNSUP),
    (dict(target=None), INVALID), (dict(target=FAKE + 2), INVALID), (dict(draft=FAKE + 2), INVALID),
    (dict(dtype=0, draft=FAKE + 1), INVALID), (dict(tokens=None), INVALID), (dict(first=None), INVALID), (dict(u=None), INVALID),
    (dict(v=None), INVALID), (dict(kept=None), INVALID), (dict(next=FAKE + 1), INVALID),
    (dict(mode=1, draft=None, ws=None), WS), (dict(mode=1, draft=None, ws=FAKE + 64), WS), (dict(mode=1, draft=None, ws_bytes=63), WS),
    (dict(n_seq=0, first=None), 0)])
def test_verify_refusals(lib, kw, code):
    assert _verify(lib.load(), **kw) == code


def test_plan_at_refusals(lib):
    L = lib.load()
    a = [FAKE, FAKE, FAKE + 2, 4, 64, 100, FAKE, 10, None, FAKE, 8, 128, FAKE, 16, FAKE, FAKE, None]
    assert L.csa2_page_plan_at(*a) == INVALID
    a[2], a[3] = FAKE, 16385
    assert L.csa2_page_plan_at(*a) == UNSUP


def test_workspace_sizes(lib):
    assert lib.csa2_workspace_size(lib.CSA2_OP_VERIFY, 6, 0) >= 48
    # a caller sizes one for its largest call: no smaller call needs more
    sizes = [lib.csa2_workspace_size(lib.CSA2_OP_EVICT, n, row) for n, row in ((1, 64), (1, 65), (2, 65), (2, 1000), (9, 1 << 20))]
    assert sizes == sorted(sizes)
    sizes = [lib.csa2_workspace_size(lib.CSA2_OP_ATTN_WEIGHT, q, n, k) for q, n, k in ((1, 1, 0), (1, 1, 512), (40, 8, 512), (8192, 100, 512))]
    assert sizes == sorted(sizes)
    for args in ((lib.CSA2_OP_ATTN_WEIGHT, 1, 1, 513), (lib.CSA2_OP_EVICT, 16385, 64, 0), (lib.CSA2_OP_VERIFY, 65536, 0, 0)):
        with pytest.raises(lib.CSA2Error):
            lib.csa2_workspace_size(*args)


# ------------------------------------------------------------------ the restatements
def test_reference_weights_are_those_of_attention():
    """The weights are the coefficients of the attention output: sum_j w_j k_j over one head alone."""
    r = np.random.default_rng(0)
    pages = np.zeros((3, 8, 288), np.uint8)
    pages[..., :256], pages[..., 256:] = r.integers(0, 256, (3, 8, 256)), r.integers(40, 60, (3, 8, 32))
    q = np.zeros((1, 64, 512))
    q[0, 5] = r.normal(size=512)
    k = R.kv_values(pages[[2, 0]].reshape(-1, 288)[:13])
    out, lse = R.attention(q[0], k, 0)
    lse_only = np.full((1, 64), np.inf)
    lse_only[0, 5] = lse[5]
    w, room, fine = K.attn_weight(q, pages, 8, np.array([[2, 0]]), [0, 1], None, [13], lse_only, 1.0, None, np.zeros(24))
    got = w.reshape(3, 8)[[2, 0]].reshape(-1)[:13]
    assert fine and np.allclose(got @ k, out[5]) and np.isclose(got.sum(), 1.0)
    assert np.count_nonzero(w) == 13


def test_reference_evict_by_hand():
    pages = np.arange(4 * 2 * 288, dtype=np.int64).astype(np.uint8).reshape(4, 2, 288)
    w = np.array([0.5, 3, 1, 2, 2, 0, 9, 9], np.float32)               # slots; table 2, 0, 1: places 0 .. 4 are slots 4 5 0 1 2
    out, w_out, n, src, fine = K.evict(pages, w, 2, np.array([[2, 0, 1]]), [5], [3], 1, None, None, np.array([[2, 0, 1]]), None, True)
    assert src == [[0, 3, 4]] and n.tolist() == [3] and fine           # weights 2 0 .5 3 | 1 (the last stays)
    assert w_out[[4, 5, 0]].tolist() == [2, 3, 1]


def test_reference_verify_by_hand():
    t = np.array([[.5, .5, 0], [.2, .3, .5], [1, 0, 0]])
    d = np.array([[.25, .75, 0], [.2, .3, .5], [0, 0, 1]])
    # token 1: .6 * .75 < .5; token 2 by row 1: .9 * .5 < .5; the last row's token
    kept, nxt, _ = K.verify(False, t, d, 3, [9, 1, 2], [0, 3], [.6, .9, 0], [.3])
    assert kept.tolist() == [3] and nxt.tolist() == [0]
    # refused: from max(p - q, 0), which is token 0's alone
    kept, nxt, _ = K.verify(False, t, d, 3, [9, 1, 2], [0, 3], [.7, .9, 0], [.99])
    assert kept.tolist() == [1] and nxt.tolist() == [0]
