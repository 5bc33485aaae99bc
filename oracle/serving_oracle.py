"""CPU oracle of the serving operators around the latent cache: TEST INFRASTRUCTURE ONLY.

Plain Python and numpy, one sequence and one page at a time, from the operators'
definitions in include/palu.h; no code is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .palu_oracle import apply_rope, decode_attention_head

__all__ = ["plan_append", "verify_drafts", "page_keys", "page_bounds", "page_scores", "select_pages",
           "decode_attention_pages"]


def plan_append(page_size, num_new, seq_lens, page_table, free_pages, num_free, n_rows):
    """One planning step on copies of its state: dict of every array after the call, and whether a
    fault (a length or rows out of range) was there to report."""
    lens, table, stack = list(seq_lens), [list(r) for r in page_table], list(free_pages)
    cap = len(table[0]) * page_size if table else 0
    slots, positions = [-1] * n_rows, [0] * n_rows
    starts, taken, fault = [0], [], False
    needs, popped, given = 0, 0, []
    for b, n in enumerate(num_new):
        row0 = starts[-1]
        starts.append(row0 + max(n, 0))
        old, new = lens[b], lens[b] + n
        if not (0 <= old <= cap and 0 <= new <= cap) or starts[-1] > n_rows:
            fault = True
            taken.append(0)
            continue
        had, has = -(-old // page_size), -(-new // page_size)
        if has > had:
            needs += has - had
            if needs > num_free:
                taken.append(0)
                continue
            for lp in range(had, has):
                table[b][lp] = stack[num_free - 1 - popped]
                popped += 1
        for lp in range(has, had):
            if 0 <= table[b][lp] < len(stack):
                given.append(table[b][lp])
            else:
                fault = True
            table[b][lp] = -1
        for j in range(max(n, 0)):
            t = old + j
            slots[row0 + j] = table[b][t // page_size] * page_size + t % page_size
            positions[row0 + j] = t
        lens[b] = new
        taken.append(n)
    left = num_free - popped
    for i, page in enumerate(reversed(given)):      # the first given back ends on top
        stack[left + i] = page
    return dict(seq_lens=lens, page_table=table, free_pages=stack, num_free=left + len(given), slot_mapping=slots,
                positions=positions, row_starts=starts, taken=taken, fault=fault)


def verify_drafts(target, draft, tokens, n, u_accept, u_sample):
    """One sequence: (output tokens, accepted).  target [D + 1][V], draft [D][V] or None, tokens [D]."""
    target = np.asarray(target, np.float64)
    V = target.shape[1]
    a = 0
    while a < n:
        x = int(tokens[a])
        q = 1.0 if draft is None else float(draft[a][x]) if 0 <= x < V else 1.0
        p = float(target[a][x]) if 0 <= x < V else 0.0
        if not float(u_accept[a]) * q < p:
            break
        a += 1

    def weights(v):
        v = np.asarray(v, np.float64)
        return np.where((v > 0) & np.isfinite(v), v, 0.0)

    p = target[a]
    if a < n:
        q = np.zeros(V) if draft is None else np.asarray(draft[a], np.float64)
        if draft is None and 0 <= int(tokens[a]) < V:
            q[int(tokens[a])] = 1.0
        with np.errstate(invalid="ignore"):
            w = weights(p - q)
        if not w.sum() > 0:
            w = weights(p)
    else:
        w = weights(p)
    total = math.fsum(w)
    out = [int(t) for t in tokens[:a]]
    if total > 0:
        at, run, pick = float(u_sample) * total, 0.0, -1
        for v in np.flatnonzero(w):
            run += w[v]
            pick = int(v)
            if run > at:
                break
        out.append(pick)
    else:
        out.append(-1)
    return out + [-1] * (target.shape[0] - len(out)), a


def page_keys(z_k, pos, B_k, head_dim, rope_base):
    """Rebuilt, rotated keys [T, W] of one group: z_k [T, r], B_k [r, W]."""
    K = np.asarray(z_k, np.float64) @ np.asarray(B_k, np.float64)
    return np.concatenate([apply_rope(K[:, c:c + head_dim], pos, rope_base)
                           for c in range(0, K.shape[1], head_dim)], axis=1)


def page_bounds(z_k, pos, B_k, head_dim, rope_base, page_size):
    """Least and largest key entries [pages, W] each, of one sequence and group."""
    k = page_keys(z_k, pos, B_k, head_dim, rope_base)
    cuts = range(0, len(k), page_size)
    return (np.array([k[t:t + page_size].min(0) for t in cuts]),
            np.array([k[t:t + page_size].max(0) for t in cuts]))


def page_scores(q, q_pos, lo, hi, group_size, rope_base):
    """Scores [G, pages] of one query q [H, d_h]; lo, hi [pages, G, W]."""
    H, d = q.shape
    qr = apply_rope(np.asarray(q, np.float64), np.full(H, q_pos), rope_base)
    out = np.empty((H // group_size, lo.shape[0]))
    for g in range(H // group_size):
        per_head = []
        for j in range(group_size):
            v, cols = qr[g * group_size + j], slice(j * d, (j + 1) * d)
            with np.errstate(invalid="ignore"):
                s = np.where(v >= 0, v * hi[:, g, cols], v * lo[:, g, cols]).sum(1)
            per_head.append(np.where(np.isnan(s), -np.inf, s))
        out[g] = np.max(per_head, axis=0)
    return out


def select_pages(scores, keep, num_first, num_last):
    """Ascending page list of one query and group from the scores of the pages it sees."""
    n = len(scores)
    fixed = {i for i in range(n) if i < num_first or i >= n - num_last}
    rest = sorted((i for i in range(n) if i not in fixed), key=lambda i: (-scores[i], i))
    return sorted(fixed | set(rest[:min(keep, n) - len(fixed)]))


def decode_attention_pages(q, q_pos, z_k, z_v, pos, B_k, B_v, group_size, rope_base, lists, page_size, causal):
    """One query over the listed pages: out [H, d_h], lse [H] and Σ p |v| [H, d_h].

    lists[g]: logical pages of head group g; causal: tokens after q_pos are left out."""
    H, d = q.shape
    out, lse, size = np.zeros((H, d)), np.full(H, -math.inf), np.zeros((H, d))
    pos = np.asarray(pos)
    T = len(pos)
    for h in range(H):
        g, j = divmod(h, group_size)
        t = np.array([t for lp in lists[g] for t in range(lp * page_size, min(T, (lp + 1) * page_size))
                      if not causal or pos[t] <= q_pos], int)
        if len(t) == 0:
            continue
        out[h], lse[h], s = decode_attention_head(h, q, q_pos, z_k[:, t], z_v[:, t], pos[t], B_k, B_v, group_size,
                                                  rope_base, return_scores=True)
        V = np.asarray(z_v[g][t], np.float64) @ np.asarray(B_v[g][:, j * d:(j + 1) * d], np.float64)
        size[h] = np.exp(s - lse[h]) @ np.abs(V)
    return out, lse, size
