"""The paged-cache operators at the ends of their numeric range, against the
64-bit restatements: heads of unlike size, long rows and their log-sum-exp,
query rows that fp32 squares cannot hold, angles of far positions."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gen import inputs as G  # noqa: E402
import paged_reference as R  # noqa: E402
from parity import ATTN_TOL_F32, row_norm_err  # noqa: E402
from test_gpu_pack_topk import _edge_rows  # noqa: E402
from test_gpu_paged import Case, _bf16, _bits, _decode_queries, _i32  # noqa: E402
from test_gpu_paged_run import _attend_rows  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    import compressed_sparse_attention_index_gb300 as c
    return c


# ------------------------------------------------------------------ heads of unlike size
def _scaled(bits, power):
    """bf16 rows times 2^power (a power a row): exact."""
    return R.round_bf16_bits(R.bf16_values(bits).astype(np.float64) * 2.0 ** np.asarray(power, np.float64)[..., None])


def _logit_room(q, k, scale=512**-0.5):
    """How far each head's logits may be off.  A logit is 32 products of 16 dims added up in fp32: each addition is off by
    a step (2^-23) of the larger of the sum so far and what is added, taken twice for products that are aligned
    before they are added."""
    a, b = torch.from_numpy(q).cuda().view(64, 32, 16), torch.from_numpy(k).cuda()
    top = torch.zeros(64, dtype=torch.float64, device="cuda")
    for c in b.split(2000):
        part = torch.einsum("hsd,nsd->hns", a, c.view(-1, 32, 16)).cumsum(-1).abs().amax((1, 2))
        step = torch.einsum("hsd,nsd->hns", a.abs(), c.view(-1, 32, 16).abs()).amax((1, 2))
        top = torch.maximum(top, torch.maximum(part, step))
    return scale * 32 * 2.0**-22 * top.cpu().numpy()


def _check_heads(c, x, out, lse, queries, rows):
    for i in rows:
        b, vis, pos, first, cnt = queries[i]
        k = R.kv_values(R.paged_rows(c.pages, c.table[b], c.page, range(vis)))
        if cnt:
            k = np.concatenate([k, R.swa_values(c.swa[b][(first + np.arange(cnt)) % c.swa_cap])])
        v = R.bf16_values(x[i]).astype(np.float64)
        o, le = R.attention(v, k, pos)
        room = _logit_room(v, k)
        # what the weights of all entries but the largest can change by: to first order where the logits are known to
        # 1/20, else by all that they may weigh
        logit = 512**-0.5 * (v @ k.T)
        logit -= logit.max(1, keepdims=True)
        w = np.exp(logit - np.log(np.exp(logit).sum(1, keepdims=True)))
        rest = np.exp(np.minimum(logit + 2 * room[:, None], 0)).sum(1) - 1
        moved = np.where(room <= 0.05, 4 * room * (w * (1 - w)).sum(1), 2 * rest)
        size = np.abs(o).max(1)
        assert np.all(np.abs(out[i] - o).max(1) <= ATTN_TOL_F32 * size + moved * np.abs(k).max()), i
        assert np.all(np.abs(lse[i] - le) <= room + 1e-5 + 2.0**-22 * np.abs(le)), i


@pytest.mark.parametrize("power", [60, 100, -60, 14])
def test_a_head_leaves_the_others_as_they_are(lib, oracle_lib, power):
    """One large or small head: the other heads keep their bits, and it has its own answer."""
    c = Case(oracle_lib, [700, 40], 64, seed=110)
    q = _decode_queries([700, 40]) + [(0, 650, 649, 0, 128)]
    want, want_l = c.run(lib, q)
    p = np.zeros((3, 64))
    p[0, 7] = p[2, 0] = p[2, 63] = power
    x = _scaled(c.q, p)
    out, lse = _attend_rows(lib, c, x, q)
    assert np.array_equal(out[p == 0], want[p == 0]) and np.array_equal(lse[p == 0], want_l[p == 0])
    _check_heads(c, x, out, lse, q, range(3))


@pytest.mark.parametrize("latent_scale,swa_scale", [(1.0, 1.0), (50.0, 1.0), (1.0, 2.0**25)])
def test_heads_of_every_size(lib, oracle_lib, latent_scale, swa_scale):
    """Heads from 2^-70 to 2^70 and a head of zeros in one query; a query of equal heads beside it."""
    c = Case(oracle_lib, [900, 300], 48, seed=111, latent_scale=latent_scale, swa_scale=swa_scale)
    q = _decode_queries([900, 300]) + [(0, 5, 4, 0, 0), (1, 299, 298, 0, 128)]
    c.run(lib, q)
    r = np.random.default_rng(5)
    x = _scaled(c.q, np.where(np.arange(4)[:, None] == 1, 0, r.integers(-70, 71, (4, 64))))
    x[0, 17] = 0
    x[3, 1], x[3, 2, 5] = 0x8000, 0x7F80               # zeros, and a head that is not finite beside the rest
    out, lse = _attend_rows(lib, c, x, q)
    assert not np.isfinite(out[3, 2]).any()
    out[3, 2], x[3, 2] = 0, 0
    o, le = _attend_rows(lib, c, x, q)
    out[3, 2], lse[3, 2] = o[3, 2], le[3, 2]
    assert np.array_equal(out, o) and np.array_equal(lse, le)
    _check_heads(c, x, out, lse, q, range(4))


def test_heads_of_unlike_size_in_many_short_rows(lib, oracle_lib):
    """Queries one after another on an SM, every third one with heads of its own sizes."""
    lens = [int(v) for v in np.random.default_rng(12).integers(1, 300, 400)]
    c = Case(oracle_lib, lens, 16, seed=112)
    q = _decode_queries(lens)
    want, want_l = c.run(lib, q)
    p = np.where(np.arange(400)[:, None] % 3 == 1, np.random.default_rng(6).integers(-40, 41, (400, 64)), 0)
    x = _scaled(c.q, p)
    out, lse = _attend_rows(lib, c, x, q)
    assert np.array_equal(out[p == 0], want[p == 0]) and np.array_equal(lse[p == 0], want_l[p == 0])
    _check_heads(c, x, out, lse, q, range(1, 400, 21))


# ------------------------------------------------------------------ query rows
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-60])
@pytest.mark.parametrize("gains", [False, True])
def test_query_rows_at_the_edges_of_their_range(lib, eps, gains):
    """Zero rows under an eps that fp32 does not hold, subnormal and huge rows, infinities and NaN, beside ordinary heads."""
    n = 5
    x = G.normal_block_bf16(130, G.S_Q, 0, 0, n * 64, 512).reshape(n, 64, 512)
    edge = _edge_rows(512)
    x[1, 3:15] = edge
    x[4, ::5][:12] = edge
    x[2, 0, 9], x[2, 1, 500], x[2, 2, 450] = 0x7F80, 0x7FC0, 0xFF80
    r = np.random.default_rng(7)
    gain = (1 + 0.2 * r.normal(size=512)).astype(np.float32)
    pos = np.array([0, 1 << 20, 77, 5, 123_457])
    out = torch.empty((n, 64, 512), dtype=torch.bfloat16, device="cuda")
    lib.csa2_qk_norm_rope(_bf16(x), 32768, torch.from_numpy(gain).cuda() if gains else None, out, None, 0, None, None, _i32(pos),
                          None, None, n, eps, None, 0, None, 0)
    there = _bf16(x)                                       # in place, the same
    lib.csa2_qk_norm_rope(there, 32768, torch.from_numpy(gain).cuda() if gains else None, there, None, 0, None, None, _i32(pos),
                          None, None, n, eps, None, 0, None, 0)
    assert np.array_equal(_bits(there), _bits(out))
    got = R.bf16_values(_bits(out)).astype(np.float64)
    ref = R.norm_rope(R.bf16_values(x), gain if gains else None, pos[:, None], eps)
    odd = np.zeros((n, 64), bool)
    odd[2, :3] = True
    # one bf16 rounding (two where a value of bf16's subnormals goes through fp32's), and fp32 arithmetic: 16 terms and 5 joins of
    # the sum (2^-20), the quotient and products (2^-22), cos and sin (2^-22) of a pair's |a| + |b|
    room = np.abs(ref)
    room[..., 448::2] += np.abs(ref[..., 449::2])
    room[..., 449::2] += np.abs(ref[..., 448::2])
    fine = np.abs(got - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-18 * room + 2.0**-133
    assert fine[~odd].all()
    # a head that is not finite: NaN where it stood (and where the rotation takes it), zeros beside an infinity
    want = np.isnan(ref[odd])
    assert np.array_equal(np.isnan(got[odd]), want) and np.all(got[odd][~want] == 0)


# ------------------------------------------------------------------ angles
def _far_rotation(y, pos, base):
    """fp64 rows rotated forward by pos, the angles to 60 digits before they are reduced; and |a| + |b| of every pair."""
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413596")
    t = np.array([float((Decimal(int(pos)) * Decimal(base) ** (Decimal(-2 * i) / 64)) % two_pi) for i in range(32)])
    a, b = y[:, 448::2].copy(), y[:, 449::2].copy()
    y[:, 448::2], y[:, 449::2] = a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)
    size = np.zeros_like(y)
    size[:, 448::2] = size[:, 449::2] = np.abs(a) + np.abs(b)
    return y, size


@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.0])
@pytest.mark.parametrize("pos", [2**31 - 1, 2**30 + 12345, 2**27 - 3, -(2**31)])
def test_latents_of_far_positions(lib, pos, base):
    """The exact value's rounding at any position: 8,192 rows have half a million rotated values, a few of which
    fall on the other side of a border with angles from a frequency of 53 bits (2^-24 at the farthest positions)."""
    n = 8192
    x = G.normal_block_bf16(140, G.S_MISC, 0, 0, n, 512)
    p = lib.default_params()
    p.rope_base = base
    out = torch.empty((n, 512), dtype=torch.bfloat16, device="cuda")
    lib.csa2_qk_norm_rope(None, 0, None, None, _bf16(x), 512, None, out, torch.full((n,), pos, dtype=torch.int32, device="cuda"), None,
                          None, n, 1e-6, None, 0, None, 0, p)
    v = R.bf16_values(x).astype(np.float64)
    ref, size = _far_rotation(v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6), pos, base)
    # a turn in 2^-64ths is off by half of one, 2^31 times at most: 2^-34 turns, 2^-31 rad; fp64's own roundings are 2^-50
    got, room = _bits(out), 2.0**-30 * size + 2.0**-48 * np.abs(ref)
    assert np.all((got == R.round_bf16_bits(ref - room)) | (got == R.round_bf16_bits(ref + room)))
    assert np.count_nonzero(got != R.round_bf16_bits(ref)) <= 8          # (as good as none: 2^-22 of the values lie so close)
@pytest.mark.parametrize("low,high", [(-5, -5), (-7, -7), (-30, -30), (20, 20), (-12, -2), (-12, 0), (-16, -2), (-25, -2), (10, 16), (15, 25),
                                      (-95, -92), (-110, -96)])
def test_queries_small_or_large_as_a_whole(lib, oracle_lib, low, high):
    """Heads of about one size, out of f16's comfortable range or on its border, beside an ordinary query."""
    c = Case(oracle_lib, [700, 300], 64, seed=113)
    q = _decode_queries([700, 300]) + [(0, 130, 129, 0, 100)]
    want, want_l = c.run(lib, q)
    p = np.random.default_rng(3).integers(low, high + 1, (3, 64))
    p[1] = 0
    x = _scaled(c.q, p)
    x[2, 8] = 0
    out, lse = _attend_rows(lib, c, x, q)
    assert np.array_equal(out[1], want[1]) and np.array_equal(lse[1], want_l[1])
    _check_heads(c, x, out, lse, q, range(3))


# ------------------------------------------------------------------ long rows, and the log-sum-exp to its figure
def _lse_room(q, k):
    """A bound of the log-sum-exp's error, over the heads of q: that of the logits; the softmax's own sums, 2^-24 an
    addition, of which an entry's numerator goes through one a chunk of 128 and 16 more; 2^-22 each for the
    exponential and the logarithm."""
    return _logit_room(q, k).max() + (len(k) / 128 + 16) * 2.0**-24 + 2 * 2.0**-22


@pytest.mark.parametrize("lens,sel", [([5000], 0), ([4000, 17, 900], 0), ([3000, 700], 500)])
def test_lse_to_its_figure(lib, oracle_lib, lens, sel):
    """Tight enough to see one entry of 5,000 missing (2e-4) or a denominator summed from rounded numerators."""
    c = Case(oracle_lib, lens, 64, seed=120)
    q = _decode_queries(lens)
    r = np.random.default_rng(2)
    pick = np.stack([np.sort(r.permutation(n)[:sel]) for n in lens]) if sel else None
    out, lse = c.run(lib, q, sel=pick)
    for i, (b, vis, pos, first, cnt) in enumerate(q):
        idx = range(vis) if pick is None else pick[i]
        k = np.concatenate([R.kv_values(R.paged_rows(c.pages, c.table[b], 64, idx)), R.swa_values(c.swa[b][(first + np.arange(cnt)) % 128])])
        v = R.bf16_values(c.q[i]).astype(np.float64)
        o, le = R.attention(v, k, pos)
        room = _lse_room(v, k) + 3 * 2.0**-24 * np.abs(le).max()          # (the result is rounded after three operations)
        assert room < 1e-4
        err = np.abs(lse[i] - le).max()
        assert err <= room, (err, room)
        assert row_norm_err(out[i], o) <= ATTN_TOL_F32


def test_a_long_row(lib):
    """100,003 entries of random records against the 64-bit form, one query of 64 heads and a short one beside it."""
    r = np.random.default_rng(121)
    n, page = 100_003, 48
    n_pages = -(-n // page) + 2
    rec = r.integers(0, 256, (n_pages * page, 288), dtype=np.uint8)
    rec[:, 256:] = r.integers(0x28, 0x38, (n_pages * page, 32))           # scales of 1/4 .. 1: latents of unit size
    table = np.stack([r.permutation(n_pages)] * 2)
    x = r.normal(size=(2, 64, 512))
    x[:, 5] *= 4.0                                                       # (a head with peaks)
    bits = R.round_bf16_bits(x)
    wsb = lib.csa2_workspace_size(lib.CSA2_OP_PAGED_ATTN, 2, 0)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((2, 64, 512), device="cuda"), torch.empty((2, 64), device="cuda")
    lib.csa2_paged_attn(_bf16(bits), torch.from_numpy(rec).cuda(), n_pages, page, _i32(table), n_pages, 2, None, 0, None, 0,
                        _i32([0, 1]), _i32([n, 300]), _i32([n - 1, 299]), _i32([0, 0]), _i32([0, 0]), 2, out, lib.CSA2_OUT_F32,
                        lse, None, ws, wsb)
    assert lib.csa2_get_device_status() == 0
    for i, vis in enumerate((n, 300)):
        j = np.arange(vis)
        k = R.kv_values(rec[table[i][j // page] * page + j % page])
        v = R.bf16_values(bits[i]).astype(np.float64)
        o, le = R.attention(v, k, vis - 1)
        assert row_norm_err(out[i].cpu().numpy(), o) <= ATTN_TOL_F32
        room = _lse_room(v, k) + 3 * 2.0**-24 * np.abs(le).max()
        assert np.abs(lse[i].cpu().numpy() - le).max() <= room


