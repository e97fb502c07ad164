"""Plain restatements, in 64 bits and Python loops, of the operators that decide what a paged cache keeps:
what tests/test_gpu_keep.py holds the kernels to."""
import numpy as np

from tests import paged_reference as R


def attn_weight(q, pages, page, table, first, sel, n_vis, lse, decay, prior, weight, scale=512 ** -0.5):
    """(weights, their bound, fine): csa2_attn_weight on fp64 queries [n_q][64][512].  The bound is that of fp32
    sums of 512 products (each of 512 roundings at most half an ulp of the running sum, all of them below the sum
    of the magnitudes, and as much again for sums that are cut instead of rounded) and of the exponential (2^-20).
    An error of d in a logit changes its exponential by exp(x + d) - exp(x) at most, which is d exp(x) for the small
    ones only: where that is infinite (logits so large that their fp32 roundings are whole units) nothing is held.
    Weights that are themselves beyond fp64 are returned as 0 with an infinite bound."""
    out, room = np.array(weight, np.float64), np.zeros(len(weight))
    fine, row = True, table.shape[1] * page
    for b in range(len(first) - 1):
        c0, c1 = int(first[b]), int(first[b + 1])
        if not 0 <= c0 <= c1 <= len(q):
            fine = False
            continue
        vis = {}
        for i in range(c0, c1):
            vis[i] = int(n_vis[i])
            if not 0 <= vis[i] <= row:
                fine, vis[i] = False, 0
        most = max(vis.values(), default=0)
        slots = np.full(most, -1, np.int64)
        for j in range(most):
            p = int(table[b, j // page])
            if 0 <= p < len(pages):
                slots[j] = p * page + j % page
        fine &= bool(np.all(slots >= 0)) or sel is not None
        on = slots >= 0
        k = np.zeros((most, 512))
        k[on] = R.kv_values(pages.reshape(-1, 288)[slots[on]])
        got, err = np.zeros(most), np.zeros(most)
        for i in range(c0, c1):
            js = np.arange(vis[i]) if sel is None else np.array([j for j in sel[i] if j >= 0], np.int64)
            fine &= bool(np.all(js < vis[i]))
            js = js[js < vis[i]]
            fine &= bool(np.all(slots[js] >= 0))
            ok = np.isfinite(lse[i]) & np.all(np.isfinite(q[i]), axis=1)
            logit = scale * (q[i][ok] @ k[js].T)
            size = scale * (np.abs(q[i][ok]) @ np.abs(k[js]).T)
            x = logit - lse[i][ok][:, None].astype(np.float64)
            d = 2 * 512 * 2.0**-24 * size + 2.0**-20 + 2.0**-22 * np.abs(lse[i][ok][:, None])
            with np.errstate(over="ignore", invalid="ignore"):
                p, e = np.exp(x), np.where(x + d > 700, np.inf, np.exp(x + d) - np.exp(x))
            np.add.at(got, js, np.where(np.isfinite(e), p, 0.0).sum(0))
            np.add.at(err, js, e.sum(0))
        s = slots[on]
        before = 0.0 if prior is None else decay * np.array(prior, np.float64)[s]
        out[s] = before + got[on]
        room[s] = err[on] + 2.0**-22 * (np.abs(before) + len(vis) * got[on])
    return out, room, fine


def evict(pages, weight, page, table, seq_len, keep, recent, dst_pages, dst_weight, dst_table, from_stride, in_place):
    """(dst_pages, dst_weight, new_len, from, fine) of csa2_evict; the last rows of from are -1."""
    pages, weight = np.array(pages), np.array(weight)
    out, w_out = (pages.copy(), weight.copy()) if in_place else (np.array(dst_pages), np.array(dst_weight))
    flat, dst = pages.reshape(-1, 288), out.reshape(-1, 288)
    new_len, source, fine = [], [], True
    for b in range(len(seq_len)):
        n, k = int(seq_len[b]), int(keep[b])
        if n < 0 or k < 0 or n > table.shape[1] * page or min(n, k) > dst_table.shape[1] * page or \
                (from_stride is not None and min(n, k) > from_stride):
            fine = False
            new_len.append(n if in_place else 0)
            source.append([])
            continue
        k = min(n, k)
        last = min(recent, k)

        def slot(t, j, n_pages):
            p = int(t[b, j // page])
            return p * page + j % page if 0 <= p < n_pages else -1
        src = [slot(table, j, len(pages)) for j in range(n)]
        fine &= k == 0 or all(s >= 0 for s in src)
        heavy = [float(weight[s]) if s >= 0 else np.nan for s in src]
        key = [-np.inf if np.isnan(x) else x for x in heavy]
        # (NaN below -inf: another key ahead of it)
        order = sorted(range(n - last), key=lambda j: (np.isnan(heavy[j]), -key[j], j))
        stay = sorted(order[:k - last]) + list(range(n - last, n))
        for r, j in enumerate(stay):
            to = slot(dst_table, r, len(out))
            fine &= to >= 0
            if to >= 0 and src[j] >= 0:
                dst[to], w_out[to] = flat[src[j]], weight[src[j]]
        if in_place:
            for j in range(k, n):
                if src[j] >= 0:
                    w_out[src[j]] = 0.0
        new_len.append(k)
        source.append(stay)
    return out, w_out, np.array(new_len), source, fine


def trim(length, new_len, page, n_pages, free, head, table):
    """(free, head, table, fine) of csa2_page_trim."""
    free, table, fine, back = np.array(free), np.array(table), True, []
    for b in range(len(length)):
        n, to = int(length[b]), int(new_len[b])
        if n < 0 or to < 0 or to > n or n > table.shape[1] * page:
            fine = False
            continue
        back += [(b, c) for c in range(-(-to // page), -(-n // page))]
    if not 0 <= head <= len(free) or len(back) > head:
        return free, head, table, False
    for i, (b, c) in enumerate(back):
        fine &= 0 <= table[b, c] < n_pages
        free[head - len(back) + i] = table[b, c]
        table[b, c] = -1
    return free, head - len(back), table, fine


def _weights(x):
    x = np.asarray(x, np.float64)
    return np.where((x >= 0) & (x <= 2.0**96), x, 0.0)       # (NaN compares false)


def verify(greedy, target, draft, vocab, tokens, first, u, v):
    """(kept, next, fine) of csa2_verify_drafts on fp64 rows, sums by math.fsum."""
    import math
    kept, nxt, fine, n_rows = [], [], True, len(target)
    for b in range(len(first) - 1):
        c0, c1 = int(first[b]), int(first[b + 1])
        if not 0 <= c0 <= c1 <= n_rows or c1 == c0:
            fine &= bool(0 <= c0 <= c1 <= n_rows)
            kept.append(0), nxt.append(-1)
            continue
        r, refused = c0, False
        while r + 1 < c1:
            x = int(tokens[r + 1])
            good = 0 <= x < vocab
            if greedy:
                row = target[r][:vocab]
                best = int(np.nanargmax(row)) if not np.all(np.isnan(row)) else -1
                stays = good and x == best
            else:
                q = 1.0 if draft is None else float(_weights(draft[r][x])) if good else 0.0
                stays = good and float(u[r]) * q < float(_weights(target[r][x]))
            if not stays:
                refused = True
                fine &= good
                break
            r += 1
        kept.append(r - c0 + 1)
        row = target[r][:vocab]
        if greedy:
            nxt.append(int(np.nanargmax(row)) if not np.all(np.isnan(row)) else -1)
            fine &= nxt[-1] >= 0
            continue
        p = _weights(row)
        w = p.copy()
        if refused and draft is not None:
            w = np.maximum(p - _weights(draft[r][:vocab]), 0.0)
        elif refused and 0 <= int(tokens[r + 1]) < vocab:
            w[int(tokens[r + 1])] = 0.0
        if not np.any(w > 0):
            w = p
        if not np.any(w > 0):
            nxt.append(-1)
            fine = False
            continue
        goal = float(v[b]) * math.fsum(w)
        some = np.flatnonzero(w > 0)
        past = np.flatnonzero(np.cumsum(w[some]) > goal)
        nxt.append(int(some[past[0]] if len(past) else some[-1]))
    return np.array(kept), np.array(nxt), fine
