"""palu_select_pages on the GPU against the CPU oracle: the lists are whole numbers and equal.

A reported score is a float32 sum over a head's channels of q'_c v_c in at most 9 steps (a chain of 4
or 4 strided terms, a join, a tree of 4 or 5): 9·2^-24 Σ|q'_c v_c|.  The rotated query is off by at
most 2^-21.5 (|q_c| + |q_pair(c)|): an angle good to 2π·2^-26 = 2^-23.3, sine and cosine to 2^-23,
two products and a sum to 2·2^-24.  With |q'_c| <= |q_c| + |q_pair(c)| the error is below
(9·2^-24 + 2^-21.5) Σ (|q_c| + |q_pair(c)|) |v_c| = 0.93·2^-20 of that sum."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200.synth import TORCH_DTYPE, WORKLOADS

pytestmark = pytest.mark.gpu
PAGE = 128
W7B = dataclasses.replace(WORKLOADS["7b_bf16_r256v128_b1_t4k"], num_heads=8)
SHAPES = {
    "7b_bf16": W7B,
    "7b_f16": dataclasses.replace(W7B, act_dtype="f16", latent_dtype="f16"),
    "norope": dataclasses.replace(W7B, rope_base=0.0),
    "tiny_f32": WORKLOADS["tiny_f32"],
    "three_heads_d40": dataclasses.replace(W7B, num_heads=6, group_size=3, head_dim=40),
    "one_head_d8": dataclasses.replace(W7B, num_heads=3, group_size=1, head_dim=8),
    "d20_f32": dataclasses.replace(WORKLOADS["tiny_f32"], head_dim=20),
    "twelve_heads": dataclasses.replace(W7B, num_heads=12, group_size=12, head_dim=64),
}


def cfg_of(w):
    return P.make_config(w.num_heads, w.head_dim, w.group_size, w.rank_k, w.rank_v, w.page_size, w.rope_base,
                         w.act_dtype, w.latent_dtype)


def make(w, lens, Q=1, seed=0, wide=None, levels=None):
    g = torch.Generator().manual_seed(seed)
    b, G, W = len(lens), w.groups, w.width
    wide = wide or max(1, max(-(-t // PAGE) for t in lens))
    pages = sum(-(-t // PAGE) for t in lens) + 2
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((b, wide), -1, dtype=torch.int32)
    at = 0
    for i, t in enumerate(lens):
        n = -(-t // PAGE)
        table[i, :n] = order[at:at + n]
        at += n
    mid, half = torch.randn((pages, G, W), generator=g), torch.rand((pages, G, W), generator=g) + 0.5
    if levels:                                    # few distinct boxes: many equal scores
        pick = torch.randint(0, levels, (pages,), generator=g)
        mid, half = mid[pick], half[pick]
    bounds = torch.stack([mid - half, mid + half], 2).to(TORCH_DTYPE[w.act_dtype])
    q = torch.randn((b, Q, w.num_heads, w.head_dim), generator=g).to(TORCH_DTYPE[w.act_dtype])
    q_pos = torch.tensor([[max(0, t - Q + j) for j in range(Q)] for t in lens], dtype=torch.int32)
    return dict(w=w, lens=lens, table=table, bounds=bounds, q=q, q_pos=q_pos, pages=pages, pos=None)


def run(c, keep, first=1, last=2, status=0, scores=True, ws=None, stream=None):
    w, cfg = c["w"], cfg_of(c["w"])
    b, Q = c["q_pos"].shape
    lists = torch.full((b, Q, w.groups, keep), 99, dtype=torch.int32, device="cuda")
    counts = torch.full((b, Q, w.groups), 99, dtype=torch.int32, device="cuda")
    sc = torch.full(lists.shape, 99.0, device="cuda") if scores else None
    if ws is None:
        ws = torch.zeros(P.palu_select_workspace_size(cfg, b, Q, c["table"].shape[1]), dtype=torch.uint8, device="cuda")
    args = [c["q"].cuda(), c["q_pos"].cuda(), c["bounds"].cuda(), None if c["pos"] is None else c["pos"].cuda(),
            c["table"].cuda(), torch.tensor(c["lens"], dtype=torch.int32, device="cuda")]
    torch.cuda.synchronize()
    P.palu_select_pages(cfg, *args, c["pages"], first, last, lists, counts, sc, ws, stream=stream)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == status
    return lists.cpu().numpy(), counts.cpu().numpy(), sc.cpu().numpy() if scores else None


def sum_of_sizes(q, box, gs):
    """Largest head's Σ (|q_c| + |q_pair(c)|) max(|lo_c|, |hi_c|) [G, pages]."""
    H, d = q.shape
    n = np.abs(q) + np.abs(np.roll(q, d // 2, axis=1))
    v = np.abs(box).max(2).reshape(len(box), H // gs, gs, d)
    return (n.reshape(H // gs, gs, d)[None] * v).sum(-1).max(-1).T


def check(c, keep, first=1, last=2, **kw):
    w = c["w"]
    lists, counts, scores = run(c, keep, first, last, **kw)
    b, Q = c["q_pos"].shape
    box = c["bounds"].double().numpy()
    for i, t in enumerate(c["lens"]):
        for j in range(Q):
            at = int(c["q_pos"][i, j])
            seen = t if Q == 1 or c["pos"] is not None else min(t, max(0, at + 1))
            n = -(-seen // PAGE)
            mine = box[c["table"][i, :n].numpy()]
            ref = S.page_scores(c["q"][i, j].double().numpy(), at, mine[:, :, 0], mine[:, :, 1], w.group_size, w.rope_base)
            size = sum_of_sizes(c["q"][i, j].double().numpy(), mine, w.group_size)
            for g in range(w.groups):
                want = S.select_pages(ref[g], keep, first, last) if n else []
                assert counts[i, j, g] == len(want)
                assert lists[i, j, g].tolist() == want + [-1] * (keep - len(want)), f"seq {i} query {j} group {g}"
                if scores is not None:
                    off = np.abs(scores[i, j, g, :len(want)] - ref[g][want])
                    assert (off <= 2.0 ** -20 * size[g][want]).all()
                    assert np.isneginf(scores[i, j, g, len(want):]).all()


@pytest.mark.parametrize("name", list(SHAPES))
def test_shapes(name):
    check(make(SHAPES[name], [5000, 1, 0, 128, 129, 2500]), 9)
    check(make(SHAPES[name], [1300, 257], Q=3, seed=1), 4)


@pytest.mark.parametrize("pages,keep", [(1, 1), (2, 3), (7, 7), (8, 7), (255, 3), (256, 64), (257, 256), (600, 100),
                                        (1025, 500), (3000, 7)])
def test_page_counts(pages, keep):
    w = dataclasses.replace(SHAPES["7b_bf16"], num_heads=2, group_size=1, head_dim=16)
    check(make(w, [pages * PAGE - 3], seed=pages), keep, 1 if keep > 1 else 0, 1)


def test_nothing_forced_and_everything_forced():
    c = make(SHAPES["7b_bf16"], [3000, 400])
    check(c, 5, 0, 0)
    check(c, 5, 5, 0)
    check(c, 5, 0, 5)
    check(c, 5, 2, 3)
    check(c, 40, 20, 20)


@pytest.mark.parametrize("levels", [1, 2, 5])
def test_equal_scores_go_to_the_lower_page(levels):
    check(make(SHAPES["7b_bf16"], [9000, 700], seed=levels, levels=levels), 13, 1, 1)


def test_queries_before_the_last_pages_and_negative_positions():
    c = make(SHAPES["7b_bf16"], [2000], Q=4)
    c["q_pos"] = torch.tensor([[-3, 0, 127, 128]], dtype=torch.int32)
    check(c, 4, 0, 1)
    c["pos"] = torch.zeros((c["pages"], PAGE), dtype=torch.int32)       # explicit positions: every page is seen
    check(c, 4, 0, 1)


def test_far_positions():
    c = make(SHAPES["7b_bf16"], [3000])
    c["q_pos"] = torch.tensor([[2 ** 31 - 1]], dtype=torch.int32)
    check(c, 6)


def test_infinite_and_nan_bounds():
    c = make(SHAPES["tiny_f32"], [1500], seed=3)
    c["bounds"][3, :, 1, 0] = float("inf")
    c["bounds"][4, :, 0, :] = float("nan")
    c["bounds"][5, 0] = float("nan")
    check(c, 5, 0, 1, scores=False)


def test_bad_pages_and_lengths_are_reported():
    c = make(SHAPES["7b_bf16"], [1000, 300])
    c["table"][0, 2] = c["pages"]
    lists, counts, _ = run(c, 4, status=7)
    assert 2 not in lists[0]
    c = make(SHAPES["7b_bf16"], [1000, 300])
    c["lens"] = [1000, -5]
    assert run(c, 4, status=7)[1][1].tolist() == [[0] * 2]


def test_one_workspace_serves_smaller_calls():
    ws = torch.zeros(P.palu_select_workspace_size(cfg_of(SHAPES["7b_bf16"]), 3, 2, 60), dtype=torch.uint8, device="cuda")
    for lens, Q in (([7000, 500, 20], 2), ([900], 1), ([7000, 7000, 7000], 2)):
        check(make(SHAPES["7b_bf16"], lens, Q=Q, wide=60), 6, ws=ws)


def test_another_stream():
    check(make(SHAPES["7b_bf16"], [7000, 500]), 6, stream=torch.cuda.Stream())


def test_scores_closer_than_float32_tells_apart():
    """Boxes that differ by one step in one channel: float32 sums tie or swap, the choice must not."""
    w = SHAPES["tiny_f32"]
    c = make(w, [PAGE * 300 - 7], seed=5, levels=1)
    g = torch.Generator().manual_seed(6)
    bits = c["bounds"].view(torch.int32)
    bits += torch.randint(-2, 3, bits.shape, generator=g, dtype=torch.int32)
    check(c, 40)
    check(c, 7, 0, 0)


def test_tiny_and_huge_scores():
    w = SHAPES["tiny_f32"]
    for scale in (1e-38, 1e-25, 1e25, 3e37):
        c = make(w, [PAGE * 200], seed=8)
        c["bounds"] *= scale
        check(c, 31, scores=False)


@pytest.mark.parametrize("name", ["tiny_f32", "d20_f32"])
def test_an_error_bound_that_overflows(name):
    """|q_c| + |q_pair(c)| past float32's range where the bounds are zero: the float32 sums stay finite
    but nothing is known of their error, and here one of them is wrong."""
    w = dataclasses.replace(SHAPES[name], rope_base=0.0, num_heads=2, group_size=1)
    c = make(w, [2 * PAGE])
    d = w.head_dim
    c["q"].fill_(1.0)
    c["q"][..., 3] = c["q"][..., 3 + d // 2] = 3e38
    c["bounds"].zero_()
    first, second = (c["bounds"][int(c["table"][0, i])] for i in (0, 1))
    first[..., 1] = 0.5
    for i, v in ((0, 2.0 ** 25), (1, 1.0), (4, -2.0 ** 25)):     # 1 in exact arithmetic, 0 in float32
        second[..., i] = v
    check(c, 1, 0, 0, scores=False)
    second[..., 1] = 0.0
    second[..., 8] = 1.0
    check(c, 1, 0, 0, scores=False)


@pytest.mark.parametrize("name", ["tiny_f32", "d20_f32"])
@pytest.mark.parametrize("far", [1e6, float("inf"), float("nan")])
def test_query_entries_that_cancel_under_rotation(name, far):
    """u cos - w sin of u = sin, w = cos in float32: the rotated entry is 0 but for roundings, and in float32
    its sign need not be float64's.  One page's box has nothing on one side of that channel and far on the
    other: the sign alone tells whether the page wins."""
    w = dataclasses.replace(SHAPES[name], group_size=1)
    d, b = w.head_dim, 40
    half = d // 2
    c = make(w, [6 * PAGE] * b, seed=2)
    rng = np.random.default_rng(4)
    c["q_pos"] = torch.from_numpy(rng.integers(1, 60000, (b, 1)).astype(np.int32))
    c["q"].zero_()
    c["bounds"].zero_()
    for i in range(b):
        for h in range(w.num_heads):
            f = int(rng.integers(0, half - 1))
            turn = int(c["q_pos"][i, 0]) * w.rope_base ** (-f / half)
            c["q"][i, 0, h, f], c["q"][i, 0, h, f + half] = math.sin(turn), math.cos(turn)
            for lp in range(6):
                box = c["bounds"][int(c["table"][i, lp]), h]
                box[:, f + half] = 1e-3 * (lp + 1)          # the last pages lead by the pair's other channel
            lp = int(rng.integers(0, 3)) + (3 if math.isnan(far) else 0)     # (NaN drops a page that leads)
            box = c["bounds"][int(c["table"][i, lp]), h]
            side = int(rng.integers(0, 2))
            box[side, f] = far if side else -far
    check(c, 2, 0, 0, scores=False)


@pytest.mark.parametrize("name,pages,levels", [("one_head_d8", 32768, 0), ("one_head_d8", 32768, 40), ("widest", 32768, 50)])
def test_the_largest_tables(name, pages, levels):
    """As many pages as the cut keeps keys of; all but a few distinct boxes have equal scores among them."""
    w = SHAPES[name] if name in SHAPES else dataclasses.replace(W7B, num_heads=64, group_size=64, page_size=128)
    real = 64 if levels else pages
    c = make(w, [PAGE * real], seed=31, levels=levels)
    g = torch.Generator().manual_seed(32)
    if levels:
        c["table"] = torch.randint(0, c["pages"], (1, pages), generator=g).to(torch.int32)
        c["lens"] = [PAGE * pages - 5]
        c["q_pos"][:] = c["lens"][0] - 1
    if name == "widest":                # (one head's oracle: the others have no part in the score)
        c["q"][:, :, 1:] = 0
        c["bounds"][..., 128:] = 0
        c["q"][:, :, 0] *= 8
    check(c, 777, scores=False)
    check(c, 5, 0, 0, scores=False)
