"""Plain restatements, in 64 bits and Python loops, of the paged-cache
operators: what tests/test_gpu_paged.py holds the kernels to.  Records are
decoded and packed by the CPU oracle."""
import numpy as np

INT_MAX = 2**31 - 1


def plan(seq_len, new_len, page, n_pages, free, head, table, swa_cap, max_tokens):
    """(desc [7][max_tokens], first, totals, table, fine) of csa2_page_plan."""
    table = np.array(table, np.int64)
    n_seq, stride = table.shape if table.size else (0, 1)
    desc = np.zeros((7, max_tokens), np.int64)
    desc[5:] = -1
    first, total, taken, fine = [0], 0, 0, True
    for b in range(n_seq):
        ln, new = int(seq_len[b]), int(new_len[b])
        if ln < 0 or new < 0 or ln + new > min(stride * page, INT_MAX):
            fine, ln, new = False, 0, 0
        have, need = -(-ln // page), -(-(ln + new) // page)
        for col in range(have, need):
            i = head + taken
            good = head >= 0 and i < len(free) and 0 <= free[i] < n_pages
            table[b, col] = free[i] if good else -1
            fine &= good
            taken += 1
        for pos in range(ln, ln + new):
            if total < max_tokens:
                cnt = min(128, swa_cap, pos + 1)
                page_id = table[b, pos // page]
                good = 0 <= page_id < n_pages
                fine &= bool(good)
                desc[:, total] = (b, pos + 1, pos, (pos + 1 - cnt) % swa_cap if swa_cap else 0, cnt,
                                  page_id * page + pos % page if good else -1,
                                  b * swa_cap + pos % swa_cap if swa_cap and pos + swa_cap >= ln + new else -1)
            else:
                fine = False
            total += 1
        first.append(total)
    return desc, np.array(first), np.array([total, taken]), table, fine


def norm_rope(x, gain, pos, eps, base=10000.0):
    """fp64 [..., 512] rows normed, scaled and rotated forward; pos broadcasts over the leading axes of x."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if gain is None else np.asarray(gain, np.float64))
    t = np.asarray(pos, np.float64)[..., None] * base ** (-2.0 * np.arange(32) / 64.0)
    a, b = y[..., 448::2].copy(), y[..., 449::2].copy()
    y[..., 448::2], y[..., 449::2] = a * np.cos(t) - b * np.sin(t), a * np.sin(t) + b * np.cos(t)
    return y


def round_bf16_bits(x):
    """fp64 -> bf16 bits, one rounding, ties to even."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore"):
        e = np.where(x == 0, -133.0, np.maximum(np.floor(np.log2(np.abs(np.where(x == 0, 1, x)))) - 7, -133.0))
    v = np.round(x / 2.0**e) * 2.0**e                 # np.round: ties to even
    bits = (v.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)      # exact: v has 8 significant bits
    return bits


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def _e4m3(b):
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0**-9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return np.where(b & 128, -v, v)


def kv_values(rec):
    """[n, 288] records -> fp64 [n, 512]."""
    rec = np.asarray(rec, np.uint8).reshape(-1, 288)
    code = np.stack([rec[:, :256] & 15, rec[:, :256] >> 4], -1).reshape(-1, 512)
    return E2M1[code] * np.repeat(_e4m3(rec[:, 256:]), 16, 1)


def swa_values(rec):
    """[n, 528] records -> fp64 [n, 512]."""
    rec = np.asarray(rec, np.uint8).reshape(-1, 528)
    return _e4m3(rec[:, :512]) * np.repeat(2.0 ** (rec[:, 512:].astype(np.float64) - 127), 32, 1)


def attention(q, k, pos, scale=512 ** -0.5, base=10000.0):
    """fp64 [64, 512] queries over latents [n, 512]: (un-rotated output, lse)."""
    q = np.asarray(q, np.float64)
    if len(k) == 0:
        return np.zeros((64, 512)), np.full(64, -np.inf)
    logit = scale * (q @ k.T)
    m = logit.max(1, keepdims=True)
    p = np.exp(logit - m)
    total = p.sum(1, keepdims=True)
    o = p @ k / total
    t = float(pos) * base ** (-2.0 * np.arange(32) / 64.0)
    a, b = o[:, 448::2].copy(), o[:, 449::2].copy()
    o[:, 448::2], o[:, 449::2] = a * np.cos(t) + b * np.sin(t), b * np.cos(t) - a * np.sin(t)
    return o, (m + np.log(total))[:, 0]


def paged_rows(pages, table_row, page, idx):
    """Records of entries idx of one sequence; those on a column that names no page are left out."""
    n_pages = pages.shape[0]
    out = [pages[table_row[j // page], j % page] for j in idx if 0 <= table_row[j // page] < n_pages]
    return np.array(out, np.uint8).reshape(-1, 288)
