"""The paged-cache entry points reject bad arguments on the host, before
anything is launched (no GPU here), and their plain restatements hold."""
import ctypes

import numpy as np
import pytest

from tests import paged_reference as R

INVALID, UNSUP, WS = 1, 2, 6
FAKE = 1 << 20                                     # never dereferenced: rejected first


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


def _plan(L, **kw):
    a = dict(seq_len=FAKE, new_len=FAKE, n_seq=4, page=64, n_pages=100, free=FAKE, n_free=10, head=None, table=FAKE,
             stride=8, cap=128, desc=FAKE, tokens=16, first=FAKE, totals=FAKE)
    a.update(kw)
    return L.csa2_page_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=-1), INVALID), (dict(page=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_free=-1), INVALID),
    (dict(stride=0), INVALID), (dict(cap=-1), INVALID), (dict(tokens=-1), INVALID), (dict(seq_len=None), INVALID),
    (dict(new_len=FAKE + 2), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(head=FAKE + 1), INVALID), (dict(desc=None), INVALID), (dict(first=None), INVALID),
    (dict(totals=None), INVALID), (dict(n_seq=16385), UNSUP), (dict(n_pages=1 << 26), UNSUP),
    (dict(cap=1 << 30), UNSUP), (dict(stride=1 << 31), UNSUP)])
def test_plan_refusals(lib, kw, code):
    assert _plan(lib.load(), **kw) == code


def _norm(L, **kw):
    a = dict(q=FAKE, q_stride=32768, q_gain=FAKE, q_out=FAKE * 64, lat=FAKE * 128, lat_stride=512, lat_gain=None,
             lat_out=FAKE * 256, pos=FAKE, slot=FAKE, swa_slot=FAKE, n=3, eps=1e-6, kv=FAKE, kv_slots=100, swa=FAKE,
             swa_slots=100, params=None)
    a.update(kw)
    return L.csa2_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(q=None, q_out=None, lat=None, lat_out=None, kv=None, swa=None), INVALID), (dict(lat=None), INVALID),
    (dict(slot=None), INVALID), (dict(swa_slot=None), INVALID), (dict(q_stride=32760), INVALID),
    (dict(q_stride=32772), INVALID), (dict(lat_stride=504), INVALID), (dict(lat_stride=516), INVALID),
    (dict(pos=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(q_gain=FAKE + 4), INVALID),
    (dict(kv=FAKE + 8), INVALID), (dict(swa=FAKE + 8), INVALID), (dict(kv_slots=-1), INVALID),
    (dict(kv_slots=1 << 31), UNSUP), (dict(n=1 << 28), UNSUP),
    (dict(q_out=FAKE + 1024), INVALID), (dict(q_out=FAKE, q_stride=32776), INVALID),      # overlapping, not in place
    (dict(lat_out=FAKE * 128 + 512), INVALID)])
def test_norm_refusals(lib, kw, code):
    assert _norm(lib.load(), **kw) == code


def test_norm_nothing_to_do(lib):
    assert _norm(lib.load(), n=0) == 0


@pytest.mark.parametrize("args,code", [
    ((7, FAKE, 10, FAKE, 4, FAKE, 0), INVALID), ((1, FAKE, 10, FAKE, 4, FAKE, 0), UNSUP),
    ((0, None, 10, FAKE, 4, FAKE, 0), INVALID), ((0, FAKE + 8, 10, FAKE, 4, FAKE, 0), INVALID),
    ((0, FAKE, -1, FAKE, 4, FAKE, 0), INVALID), ((0, FAKE, 10, None, 4, FAKE, 0), INVALID),
    ((0, FAKE, 10, FAKE, -4, FAKE, 0), INVALID), ((0, FAKE, 10, FAKE, 4, FAKE + 4, 0), INVALID),
    ((0, FAKE, 10, FAKE, 4, FAKE, 2), INVALID), ((2, None, 10, None, 0, None, 1), 0)])
def test_read_refusals(lib, args, code):
    assert lib.load().csa2_cache_read(*args, None) == code


def _attn(L, **kw):
    a = dict(q=FAKE, pages=FAKE, n_pages=100, page=64, table=FAKE, stride=8, n_seq=2, sel=None, sel_stride=0,
             swa=FAKE, cap=128, q_seq=FAKE, n_vis=FAKE, pos=FAKE, first=FAKE, cnt=FAKE, n_q=2, out=FAKE, dt=0,
             lse=None, params=None, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return L.csa2_paged_attn(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_q=-1), INVALID), (dict(n_seq=0), INVALID), (dict(n_pages=0), INVALID), (dict(page=0), INVALID),
    (dict(stride=0), INVALID), (dict(cap=-1), INVALID), (dict(dt=2), INVALID), (dict(sel=FAKE, sel_stride=0), INVALID),
    (dict(sel=FAKE, sel_stride=513), INVALID), (dict(n_q=65536), UNSUP), (dict(stride=1 << 31), UNSUP),
    (dict(q=FAKE + 8), INVALID), (dict(pages=FAKE + 16), INVALID), (dict(table=None), INVALID),
    (dict(swa=None), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(out=FAKE + 8), INVALID), (dict(pos=None), INVALID),
    (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(ws_bytes=1024), WS), (dict(n_q=0, q=None), 0)])
def test_attn_refusals(lib, kw, code):
    assert _attn(lib.load(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_pages=1 << 16, page=1 << 15), UNSUP),                               # slots of 32 bits
    (dict(n_q=65535, n_pages=10, page=64, stride=1 << 15), UNSUP),              # 65,535 rows of 2^21 entries: chunks of 32 bits
    (dict(n_q=200, page=1 << 20, stride=1 << 30), UNSUP)])                      # (the product of both behind 64 bits' half)
def test_attn_limits(lib, kw, code):
    assert _attn(lib.load(), **kw) == code


def test_params_other_than_the_constants(lib):
    p = lib.default_params()
    p.heads = 32
    assert _norm(lib.load(), params=ctypes.byref(p)) == UNSUP
    assert _attn(lib.load(), params=ctypes.byref(p)) == UNSUP


def test_workspace_is_the_same_for_every_call(lib):
    a = lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, 0, 0, 0)
    assert a == lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, 65535, 1 << 20, 7) and a > 0


def test_paged_cache_refuses_what_does_not_fit():
    import torch
    from compressed_sparse_attention_index_gb300.decode import PagedCache
    c = PagedCache(3, 8, 16, 64, 5, device="cpu")
    q, lat = torch.zeros((5, 64, 512), dtype=torch.bfloat16), torch.zeros((5, 512), dtype=torch.bfloat16)
    for new in (torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros((3, 2), dtype=torch.int32)[:, 0]):
        with pytest.raises(ValueError):
            c.plan(new)
    for a, b in ((q[:4], lat), (q, lat[:4]), (q.float(), lat), (q, lat.float()), (q.transpose(1, 2), lat), (q, lat[:, ::2]),
                 (q.transpose(0, 1), lat), (q[:, :32], lat)):
        with pytest.raises(ValueError):
            c.write(a, b)
    for gain in (torch.ones(256), torch.ones(512, dtype=torch.float64), torch.ones(1024)[::2]):
        with pytest.raises(ValueError):
            c.write(q, lat, gain)
    for sel in (torch.zeros((4, 8), dtype=torch.int32), torch.zeros((5, 8)), torch.zeros((5, 16), dtype=torch.int32)[:, ::2]):
        with pytest.raises(ValueError):
            c.attend(sel)
    slots = torch.zeros(6, dtype=torch.int32)
    for out in (torch.zeros((5, 512)), torch.zeros((6, 512), dtype=torch.float16), torch.zeros((6, 1024))[:, ::2]):
        with pytest.raises(ValueError):
            c.read(slots, out)
    with pytest.raises(ValueError):
        c.read(slots.long(), torch.zeros((6, 512)))


# ------------------------------------------------------------------ the restatements themselves
def test_rounding_matches_the_library_conversion():
    import torch
    x = np.concatenate([np.random.default_rng(0).normal(size=4000) * 10.0 ** np.random.default_rng(1).integers(-30, 30, 4000),
                        [0.0, -0.0, 1 + 2.0**-8, 1 + 3 * 2.0**-8, 2.0**-133, 2.0**-134]]).astype(np.float32)
    want = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(R.round_bf16_bits(x.astype(np.float64)), want)


def test_decoding_matches_the_oracle(oracle_lib):
    from gen import inputs as G
    x = G.normal_block_bf16(5, G.S_MISC, 0, 0, 40, 512)
    kv, swa = oracle_lib.pack_kv(x), oracle_lib.pack_swa(x)
    v = R.bf16_values(x).astype(np.float64)
    # within half a step of the format: FP4 spacing is at most 1/3 of the value's binade top, FP8 2^-4
    assert np.abs(R.kv_values(kv) - v).max() <= np.abs(v).max() / 6 and np.abs(R.swa_values(swa) - v).max() <= 2.0**-4 * np.abs(v).max()
    o, lse = R.attention(np.zeros((64, 512)), R.kv_values(kv), 0)
    assert np.allclose(o, R.kv_values(kv).mean(0)) and np.allclose(lse, np.log(40))


def test_rotation_is_undone():
    x = np.random.default_rng(2).normal(size=(3, 512))
    y = R.norm_rope(x, None, [5, 70_000, 1_000_003], 1e-6)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    for i, p in enumerate((5, 70_000, 1_000_003)):
        o, _ = R.attention(np.zeros((64, 512)), y[i:i + 1], p)       # one entry: its latent, un-rotated
        assert np.allclose(o[0], n[i], atol=1e-9)


def test_plan_by_hand():
    desc, first, totals, table, fine = R.plan([3, 0, 4], [2, 0, 1], 4, 9, [7, 8, 5], 0, np.full((3, 3), 1), 4, 5)
    assert fine and first.tolist() == [0, 2, 2, 3] and totals.tolist() == [3, 2]
    assert table[0].tolist() == [1, 7, 1] and table[2].tolist() == [1, 8, 1]
    assert desc[:, 0].tolist() == [0, 4, 3, 0, 4, 7, 3] and desc[:, 1].tolist() == [0, 5, 4, 1, 4, 28, 0]
    assert desc[:, 2].tolist() == [2, 5, 4, 1, 4, 32, 8] and desc[:, 3].tolist() == [0, 0, 0, 0, 0, -1, -1]
