"""Pins of the serving operators' oracle: closed forms, brute force and invariants.  CPU only."""
import itertools
import random

import numpy as np
import pytest

from oracle import palu_oracle as O
from oracle import serving_oracle as S


def _state(rng, batch, P, num_pages, wide):
    lens = [rng.randint(0, wide * P // 2) for _ in range(batch)]
    pages = rng.sample(range(num_pages), num_pages)
    table = [[-1] * wide for _ in range(batch)]
    for b, t in enumerate(lens):
        for lp in range(-(-t // P)):
            table[b][lp] = pages.pop()
    return lens, table, pages + [-1] * (num_pages - len(pages)), len(pages)


@pytest.mark.parametrize("seed", range(20))
def test_plan_keeps_every_page_once(seed):
    rng = random.Random(seed)
    P, wide, batch = 8, 6, rng.randint(1, 7)
    lens, table, stack, free = _state(rng, batch, P, 60, wide)
    new = [rng.randint(-t, wide * P - t) for t in lens]
    free = rng.randint(0, free)
    owned = sorted([p for r in table for p in r if p >= 0] + stack[:free])
    r = S.plan_append(P, new, lens, table, stack, free, sum(max(n, 0) for n in new))
    assert not r["fault"]
    assert sorted([p for row in r["page_table"] for p in row if p >= 0] + r["free_pages"][:r["num_free"]]) == owned
    for b, t in enumerate(r["seq_lens"]):
        assert t == lens[b] + r["taken"][b]
        assert [p >= 0 for p in r["page_table"][b]] == [lp < -(-t // P) for lp in range(wide)]
        for j in range(max(new[b], 0)):
            row = r["row_starts"][b] + j
            if r["taken"][b] == 0:
                assert (r["slot_mapping"][row], r["positions"][row]) == (-1, 0)
            else:
                at = lens[b] + j
                assert r["positions"][row] == at
                assert r["slot_mapping"][row] == r["page_table"][b][at // P] * P + at % P


def test_plan_dropping_what_was_appended_restores_the_state():
    rng = random.Random(3)
    lens, table, stack, free = _state(rng, 5, 16, 80, 8)
    new = [9, 0, 40, 17, 1]
    r = S.plan_append(16, new, lens, table, stack, free, 67)
    assert r["taken"] == new
    back = S.plan_append(16, [-n for n in new], r["seq_lens"], r["page_table"], r["free_pages"], r["num_free"], 0)
    assert (back["seq_lens"], back["page_table"], back["free_pages"][:free], back["num_free"]) == \
        (lens, table, stack[:free], free)


def test_verify_output_is_distributed_as_the_target():
    """Integrated over drafts ~ q and a fine grid of both random numbers, the first output token
    follows p: P(x) = q(x) min(1, p(x)/q(x)) + P(refused) (p - q)+ / Σ (p - q)+ = p(x)."""
    p = np.array([[0.5, 0.25, 0.125, 0.125], [0.25, 0.25, 0.25, 0.25]])
    q = np.array([[0.125, 0.5, 0.25, 0.125]])
    n = 64
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(4)
    for x in range(4):
        for ua, us in itertools.product(grid, grid):
            out, a = S.verify_drafts(p, q, [x], 1, [ua], us)
            got[out[0]] += q[0, x] / n ** 2
            assert (a == 1) == (out[0] == x and out[1] >= 0)
    np.testing.assert_allclose(got, p[0], atol=1.0 / n)


def test_verify_equal_distributions_accept_everything():
    p = np.full((3, 4), 0.25)
    out, a = S.verify_drafts(p, p[:2], [1, 3], 2, [0.999, 0.5], 0.6)
    assert (out, a) == ([1, 3, 2], 2)


def test_verify_certain_draft_and_empty_rows():
    p = np.array([[0.2, 0.8], [0.5, 0.5]])
    assert S.verify_drafts(p, None, [0], 1, [0.1], 0.0) == ([0, 0], 1)
    assert S.verify_drafts(p, None, [0], 1, [0.2], 0.0) == ([1, -1], 0)      # 0.2·1 < 0.2 fails
    assert S.verify_drafts(np.zeros((2, 2)), None, [0], 1, [0.5], 0.3) == ([-1, -1], 0)
    # p <= q everywhere: the draw falls back to p
    assert S.verify_drafts([[0.1, 0.2], [1, 0]], [[0.5, 0.5]], [0], 1, [0.9], 0.5) == ([1, -1], 0)


def test_bounds_contain_every_key_and_scores_bound_every_token():
    rng = np.random.default_rng(0)
    T, r, d, gs, P = 45, 16, 8, 2, 16
    z, B, pos = rng.standard_normal((1, T, r)), rng.standard_normal((1, r, gs * d)), np.arange(T)
    q = rng.standard_normal((gs, d))
    lo, hi = S.page_bounds(z[0], pos, B[0], d, 100.0, P)
    k = S.page_keys(z[0], pos, B[0], d, 100.0)
    for p in range(3):
        assert (k[p * P:(p + 1) * P] >= lo[p]).all() and (k[p * P:(p + 1) * P] <= hi[p]).all()
        assert (k[p * P:(p + 1) * P] == lo[p]).any(0).all()
    score = S.page_scores(q, T - 1, lo[:, None], hi[:, None], gs, 100.0)[0]
    for h in range(gs):
        s = O.decode_attention_head(h, q, T - 1, z, z, pos, B, B, gs, 100.0, return_scores=True)[2] * d ** 0.5
        for p in range(3):
            assert s[p * P:(p + 1) * P].max() <= score[p] + 1e-12


def test_select_is_brute_force_top_k():
    rng = random.Random(1)
    for _ in range(200):
        n = rng.randint(1, 12)
        scores = [rng.choice([0.0, 1.0, 2.0, -np.inf, rng.random()]) for _ in range(n)]
        first, last = rng.randint(0, 2), rng.randint(0, 2)
        keep = rng.randint(max(1, first + last), 8)
        got = S.select_pages(scores, keep, first, last)
        assert len(got) == min(keep, n) and got == sorted(set(got))
        fixed = [i for i in range(n) if i < first or i >= n - last]
        assert set(fixed) <= set(got)
        for i in set(range(n)) - set(got):
            for j in set(got) - set(fixed):
                assert (scores[j], -j) > (scores[i], -i)


def test_attention_over_all_pages_is_the_dense_step():
    rng = np.random.default_rng(2)
    T, r, d, gs, H = 37, 16, 8, 2, 4
    z_k, z_v = rng.standard_normal((2, T, r)), rng.standard_normal((2, T, r))
    B_k, B_v = rng.standard_normal((2, r, gs * d)), rng.standard_normal((2, r, gs * d))
    q = rng.standard_normal((H, d))
    out, lse, _ = S.decode_attention_pages(q, T - 1, z_k, z_v, np.arange(T), B_k, B_v, gs, 1e4, [range(5)] * 2, 8, False)
    ref, ref_lse = O.decode_attention(q, T - 1, z_k, z_v, np.arange(T), B_k, B_v, gs, 1e4)
    np.testing.assert_allclose(out, ref, rtol=1e-12)
    np.testing.assert_allclose(lse, ref_lse, rtol=1e-12)
