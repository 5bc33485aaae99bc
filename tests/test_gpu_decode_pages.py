"""palu_decode_attn_pages on the GPU against the CPU oracle, on every decode path.

Error bounds.  A 16-bit result carries its final rounding, half a step: 2^-8 (bf16) or 2^-11 (f16) of
its value.  Before it, a score is off by at most Σ|q||k|·2^-20 / √d for the hardware sine and cosine,
twice (query and key) and 4e-5 for |q|, |k| <= 15, so a weight by 8e-5 relative; the weights' split in
two 16-bit numbers by 2^-16: together 1.2e-4 Σ p|v|.  In float32 angles are correct to 2^-23 and the
bound is 2e-5 Σ p|v|.  Log-sum-exps are off by at most the score error, 1e-4 (1e-5 in float32).
"""
import dataclasses
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from palu_testlib import build_pools, build_ranked_pools, make_decode_case, make_ranked_case
from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200.synth import TORCH_DTYPE, WORKLOADS, normal_tensor

pytestmark = pytest.mark.gpu
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SUM = {"bf16": 1.2e-4, "f16": 1.2e-4, "f32": 2e-5}
LSE = {"bf16": 1e-4, "f16": 1e-4, "f32": 1e-5}


def w7b(**kw):
    return dataclasses.replace(WORKLOADS["7b_bf16_r256v128_b1_t4k"], num_heads=8, **kw)


CASES = {
    "bf16": (w7b(), 2),
    "f16_r256": (w7b(act_dtype="f16", latent_dtype="f16", rank_v=256), 2),
    "two_heads_r64": (w7b(group_size=2, rank_k=64), 2),
    "norope": (w7b(rope_base=0.0), 3),
    "norope_f16_r256": (w7b(rope_base=0.0, act_dtype="f16", latent_dtype="f16", rank_v=256), 3),
    "int4_f16": (dataclasses.replace(WORKLOADS["7b_int4_r256_b8_t32k"], num_heads=8), 2),
    "int4_bf16": (dataclasses.replace(WORKLOADS["7b_int4_r256_b8_t32k"], num_heads=8, act_dtype="bf16"), 2),
    "tiny_f32": (WORKLOADS["tiny_f32"], 1),
    "odd_heads": (dataclasses.replace(WORKLOADS["tiny_f32"], num_heads=6, group_size=3, head_dim=40, act_dtype="bf16",
                                      latent_dtype="bf16", page_size=24), 1),
}


def pick_lists(case, Q, keep, seed=0, last=True):
    """Random ascending lists [b][Q][G] of at most `keep` pages."""
    rng = np.random.default_rng(seed)
    out = []
    for t in case.seq_lens:
        n = -(-t // case.w.page_size)
        out.append([[sorted(rng.permutation(n)[:min(n, rng.integers(1, keep + 1))].tolist()) if n else []
                     for _ in range(case.w.groups)] for _ in range(Q)])
        if last and n:
            for row in out[-1]:
                for g in range(0, case.w.groups, 2):
                    row[g] = sorted(set(row[g][:keep - 1]) | {n - 1})
    return out


def run(case, pools, q, q_pos, lists, keep, num_splits=0, status=0, ranks=(None, None), B=None, table=None, stream=None,
        lse=True):
    w, cfg = case.w, case.cfg
    b, Q = q_pos.shape
    flat = np.full((b, Q, w.groups, keep), -1, np.int32)
    counts = np.zeros((b, Q, w.groups), np.int32)
    for i in range(b):
        for j in range(Q):
            for g in range(w.groups):
                flat[i, j, g, :len(lists[i][j][g])] = lists[i][j][g]
                counts[i, j, g] = len(lists[i][j][g])
    out = torch.full((b, Q, w.num_heads, w.head_dim), 9.0, dtype=TORCH_DTYPE[w.act_dtype], device="cuda")
    ls = torch.full((b, Q, w.num_heads), 9.0, device="cuda") if lse else None
    ws = torch.zeros(P.palu_decode_pages_workspace_size(cfg, b, Q, keep, num_splits, *ranks), dtype=torch.uint8,
                     device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    args = (q.cuda(), dev(q_pos), pools["zk"], pools["zv"], pools["zks"], pools["zvs"], pools["pos"],
            dev(case.page_table if table is None else table), torch.tensor(case.seq_lens, dtype=torch.int32, device="cuda"),
            dev(flat), dev(counts), case.num_pages, case.B_k.cuda(), case.B_v.cuda(), out, ls, ws)
    torch.cuda.synchronize()
    P.palu_decode_attn_pages(cfg, *args, num_splits, *ranks, stream=stream)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == status
    return out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None


def queries(case, Q, seed=5):
    w = case.w
    q = normal_tensor(seed, "q_pages", (len(case.seq_lens), Q, w.num_heads, w.head_dim), w.act_dtype)
    q_pos = np.array([[int(case.positions(i)[max(T - Q + j, 0)]) if T else j for j in range(Q)]
                      for i, T in enumerate(case.seq_lens)], np.int32)
    return q, q_pos


def compare(case, out, lse, q, q_pos, lists, inputs):
    w = case.w
    b, Q = q_pos.shape
    for i in range(b):
        zk, zv, Bk, Bv = inputs(i)
        for j in range(Q):
            ref, rl, size = S.decode_attention_pages(q[i, j].double().numpy(), q_pos[i, j], zk, zv, case.positions(i),
                                                     Bk, Bv, w.group_size, w.rope_base, lists[i][j], w.page_size, Q > 1)
            off = np.abs(out[i, j] - ref)
            assert (off <= HALF_STEP[w.act_dtype] * np.abs(ref) + SUM[w.act_dtype] * size + 1e-30).all(), \
                f"seq {i} query {j}: {off.max():.3e} of {np.abs(ref).max():.3e}"
            if lse is not None:
                empty = np.isneginf(rl)
                assert (np.isneginf(lse[i, j]) == empty).all()
                np.testing.assert_allclose(lse[i, j][~empty], rl[~empty], rtol=0, atol=LSE[w.act_dtype])


def uniform(case):
    Bk, Bv = case.B_k.double().numpy(), case.B_v.double().numpy()
    return lambda i: (*case.oracle_latents(i), Bk, Bv)


@pytest.mark.parametrize("Q", [1, 3])
@pytest.mark.parametrize("name", list(CASES))
def test_listed_pages(name, Q):
    w, kind = CASES[name]
    case = make_decode_case(w, [300, 0, 1, 128, 1000])
    assert P.palu_decode_kernel_kind(case.cfg) == kind
    q, q_pos = queries(case, Q)
    pools = build_pools(case)
    for splits in (0, 1, 3):
        lists = pick_lists(case, Q, 5, seed=splits)
        compare(case, *run(case, pools, q, q_pos, lists, 5, splits), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16", "tiny_f32"])
def test_explicit_positions(name):
    case = make_decode_case(CASES[name][0], [300, 129, 700], explicit_positions=True)
    q, q_pos = queries(case, 2)
    lists = pick_lists(case, 2, 4)
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 4), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16", "odd_heads"])
def test_every_page_listed_is_the_dense_step(name):
    case = make_decode_case(CASES[name][0], [515, 77])
    q, q_pos = queries(case, 1)
    lists = [[[list(range(-(-t // case.w.page_size)))] * case.w.groups] for t in case.seq_lens]
    keep = max(len(x[0][0]) for x in lists)
    compare(case, *run(case, build_pools(case), q, q_pos, lists, keep), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16"])
def test_long_lists(name):
    """Lists that wrap every ring and both TMEM slots many times, one split and many."""
    case = make_decode_case(dataclasses.replace(CASES[name][0], num_heads=4), [40 * 128 - 5])
    q, q_pos = queries(case, 1)
    pools = build_pools(case)
    lists = [[[[p for p in range(40) if p % 5 != 1]]]]
    for splits in (1, 7, 32):
        compare(case, *run(case, pools, q, q_pos, lists, 32, splits), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "tiny_f32"])
def test_queries_that_see_none_of_their_pages(name):
    case = make_decode_case(CASES[name][0], [600])
    q, _ = queries(case, 3)
    q_pos = np.array([[100, 255, 599]], np.int32)
    lists = [[[[1, 3]] * case.w.groups, [[2]] * case.w.groups, [[0, 4]] * case.w.groups]]
    if name == "tiny_f32":
        assert case.w.page_size == 128
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 2), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope"])
def test_ranks_per_group(name):
    ranks_k, ranks_v = [128, 256], [128, 256]
    case = make_ranked_case(CASES[name][0], ranks_k, ranks_v, [300, 700], nq=2)
    q, q_pos = case.q, case.q_pos
    lists = [[[[0, 2], [1]], [[0], [0, 2]]], [[[5], [0, 3, 5]], [[1, 2], [4]]]]
    out, lse = run(case, build_ranked_pools(case), q, q_pos, lists, 3, ranks=(ranks_k, ranks_v))
    w = case.w
    for i in range(2):
        zk, zv, Bk, Bv = case.oracle_inputs(i)
        for j in range(2):
            for g in range(2):
                hs = slice(g * 4, g * 4 + 4)
                ref, rl, size = S.decode_attention_pages(q[i, j, hs].double().numpy(), q_pos[i, j], zk[g][None],
                                                         zv[g][None], case.positions(i), Bk[g][None], Bv[g][None], 4,
                                                         w.rope_base, [lists[i][j][g]], w.page_size, True)
                off = np.abs(out[i, j, hs] - ref)
                assert (off <= HALF_STEP[w.act_dtype] * np.abs(ref) + SUM[w.act_dtype] * size).all()
                np.testing.assert_allclose(lse[i, j, hs], rl, rtol=0, atol=LSE[w.act_dtype])


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16", "tiny_f32"])
def test_bad_lists_are_reported(name):
    case = make_decode_case(CASES[name][0], [600])
    q, q_pos = queries(case, 1)
    pools = build_pools(case)
    G = case.w.groups
    for bad in ([1, 1], [3, 2], [0, 5], [-1, 2]):
        run(case, pools, q, q_pos, [[[bad] * G]], 2, status=7)
    table = case.page_table.copy()
    table[0, 1] = -7
    run(case, pools, q, q_pos, [[[[1, 2]] * G]], 2, status=7, table=table)
    good = [[[[0, 4]] * G]]                                  # and the next call is whole again
    compare(case, *run(case, pools, q, q_pos, good, 2), q, q_pos, good, uniform(case))


def test_another_stream_and_no_lse():
    case = make_decode_case(CASES["bf16"][0], [300, 700])
    q, q_pos = queries(case, 1)
    lists = pick_lists(case, 1, 3)
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 3, stream=torch.cuda.Stream(), lse=False), q, q_pos,
            lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "tiny_f32"])
def test_rows_behind_the_last_token_are_not_read(name):
    case = make_decode_case(CASES[name][0], [133, 7])
    q, q_pos = queries(case, 1)
    pools = build_pools(case)
    w = case.w
    T = TORCH_DTYPE[w.latent_dtype]
    for pool, rank in (("zk", w.rank_k), ("zv", w.rank_v)):
        raw = pools[pool].view(case.num_pages, w.groups, rank * T.itemsize // 128, w.page_size, 128)
        for i, t in enumerate(case.seq_lens):
            page = int(case.page_table[i, t // w.page_size])
            junk = raw[page, :, :, t % w.page_size:].contiguous().view(T)
            junk[..., 0::2], junk[..., 1::2] = float("nan"), float("inf")
            raw[page, :, :, t % w.page_size:] = junk.view(torch.uint8)
    lists = [[[[0, 1]] * w.groups], [[[0]] * w.groups]]
    compare(case, *run(case, pools, q, q_pos, lists, 2), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "tiny_f32"])
def test_tokens_after_the_query_may_hold_anything(name):
    """NaN and infinities in the latents of the drafts behind a query do not reach its result."""
    case = make_decode_case(CASES[name][0], [260])
    w = case.w
    q, _ = queries(case, 3)
    q_pos = np.array([[126, 255, 256]], np.int32)            # the last token of a page but one, the last, the first
    pools = build_pools(case)
    T = TORCH_DTYPE[w.latent_dtype]
    lists = [[[[0, 1]] * w.groups, [[1]] * w.groups, [[0, 2]] * w.groups]]
    for t in range(257, 260):
        for pool, rank in (("zk", w.rank_k), ("zv", w.rank_v)):
            raw = pools[pool].view(case.num_pages, w.groups, rank * T.itemsize // 128, w.page_size, 128)
            junk = raw[int(case.page_table[0, t // w.page_size]), :, :, t % w.page_size].contiguous().view(T)
            junk[..., 0::2], junk[..., 1::2] = float("nan"), float("inf")
            raw[int(case.page_table[0, t // w.page_size]), :, :, t % w.page_size] = junk.view(torch.uint8)
    compare(case, *run(case, pools, q, q_pos, lists, 2), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "int4_f16", "norope"])
def test_timeout_reports_and_recovers(name):
    case = make_decode_case(CASES[name][0], [600])
    q, q_pos = queries(case, 1)
    pools = build_pools(case)
    lists = [[[[0, 2, 4]] * case.w.groups]]
    P.palu_debug_timeout_test(1 << 20, stall=True)
    try:
        run(case, pools, q, q_pos, lists, 3, status=6)
    finally:
        P.palu_debug_timeout_test()
    compare(case, *run(case, pools, q, q_pos, lists, 3), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["int4_f16", "int4_bf16"])
def test_scales_behind_the_last_token_are_not_read(name):
    case = make_decode_case(CASES[name][0], [133, 7])
    q, q_pos = queries(case, 1)
    pools = build_pools(case)
    w = case.w
    for pool in ("zks", "zvs"):
        raw = pools[pool].view(torch.float16).view(case.num_pages, w.groups, w.page_size, -1)
        for i, t in enumerate(case.seq_lens):
            page, rest = int(case.page_table[i, t // w.page_size]), raw[:, :, t % w.page_size:]
            rest[page, :, 0::2], rest[page, :, 1::2] = float("nan"), float("inf")
    lists = [[[[0, 1]] * w.groups], [[[0]] * w.groups]]
    compare(case, *run(case, pools, q, q_pos, lists, 2), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16", "tiny_f32"])
def test_calls_that_follow_at_once_share_a_workspace(name):
    """Calls of other sizes behind one another on a stream, nothing waited for: each as on its own."""
    case = make_decode_case(CASES[name][0], [900, 0, 1, 400])
    pools, cfg, w = build_pools(case), case.cfg, case.w
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    table, lens = dev(case.page_table), torch.tensor(case.seq_lens, dtype=torch.int32, device="cuda")
    Bk, Bv = case.B_k.cuda(), case.B_v.cuda()
    ws = torch.zeros(P.palu_decode_pages_workspace_size(cfg, 4, 4, 7), dtype=torch.uint8, device="cuda")
    calls = []
    for n in range(12):
        Q, keep = (1, 4, 2)[n % 3], (7, 1, 3)[n % 3]
        q, q_pos = queries(case, Q, seed=n)
        lists = pick_lists(case, Q, keep, seed=n)
        if n % 4 == 3:
            lists = [[[[]] * w.groups for _ in range(Q)] for _ in lists]     # nothing listed at all
        flat = np.full((4, Q, w.groups, keep), -1, np.int32)
        counts = np.zeros((4, Q, w.groups), np.int32)
        for i, j, g in np.ndindex(4, Q, w.groups):
            flat[i, j, g, :len(lists[i][j][g])] = lists[i][j][g]
            counts[i, j, g] = len(lists[i][j][g])
        out = torch.full((4, Q, w.num_heads, w.head_dim), 9.0, dtype=TORCH_DTYPE[w.act_dtype], device="cuda")
        lse = torch.full((4, Q, w.num_heads), 9.0, device="cuda")
        calls.append((q, q_pos, lists, q.cuda(), dev(q_pos), dev(flat), dev(counts), out, lse))
    torch.cuda.synchronize()
    for _, _, _, q, q_pos, flat, counts, out, lse in calls:
        P.palu_decode_attn_pages(cfg, q, q_pos, pools["zk"], pools["zv"], pools["zks"], pools["zvs"], pools["pos"], table,
                                 lens, flat, counts, case.num_pages, Bk, Bv, out, lse, ws)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == 0
    for q, q_pos, lists, *_, out, lse in calls:
        compare(case, out.double().cpu().numpy(), lse.double().cpu().numpy(), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("Q", [1, 2])
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("rank_k", [64, 320, 384, 448, 512])
def test_norope_at_every_number_of_key_chunks(rank_k, act, Q):
    """A list's first tile has more latent chunks than the ring has stages from key rank 448 on."""
    w = w7b(rope_base=0.0, rank_k=rank_k, act_dtype=act, latent_dtype=act)
    case = make_decode_case(w, [300, 0, 1, 900])
    assert P.palu_decode_kernel_kind(case.cfg) == 3
    q, q_pos = queries(case, Q)
    lists = pick_lists(case, Q, 5, seed=rank_k)
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 5), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("ranks_k", [[128, 512], [448, 64]])
def test_norope_ranks_per_group_up_to_the_largest(ranks_k):
    case = make_ranked_case(w7b(rope_base=0.0), ranks_k, [128, 128], [300, 700], nq=2)
    lists = [[[[0, 2], [1]], [[0], [0, 2]]], [[[5], [0, 3, 5]], [[1, 2], [4]]]]
    out, lse = run(case, build_ranked_pools(case), case.q, case.q_pos, lists, 3, ranks=(ranks_k, [128, 128]))
    w = case.w
    for i in range(2):
        zk, zv, Bk, Bv = case.oracle_inputs(i)
        for j in range(2):
            for g in range(2):
                hs = slice(g * 4, g * 4 + 4)
                ref, rl, size = S.decode_attention_pages(case.q[i, j, hs].double().numpy(), case.q_pos[i, j], zk[g][None],
                                                         zv[g][None], case.positions(i), Bk[g][None], Bv[g][None], 4,
                                                         w.rope_base, [lists[i][j][g]], w.page_size, True)
                off = np.abs(out[i, j, hs] - ref)
                assert (off <= HALF_STEP[w.act_dtype] * np.abs(ref) + SUM[w.act_dtype] * size).all()
                np.testing.assert_allclose(lse[i, j, hs], rl, rtol=0, atol=LSE[w.act_dtype])


def one_channel(name, T, a, v, **kw):
    """A case whose scores are exact: latent entry 0 of token t is a[t], it reaches channel 40 of every
    head alone, where no angle is left (RoPE's frequencies vanish from channel 32 on at this base), and
    the query is 8 there.  Value channel j of every head is latent entry j, v[t][j]."""
    w = dataclasses.replace(CASES[name][0], num_heads=CASES[name][0].group_size, **kw)
    if w.rope_base:
        w = dataclasses.replace(w, rope_base=3e38)
    case = make_decode_case(w, [T])
    q, q_pos = queries(case, 1)
    q.zero_()
    q[..., 40] = 8.0
    case.B_k.zero_()
    case.B_v.zero_()
    for h in range(w.group_size):
        case.B_k[0, 0, h * 128 + 40] = 1.0
        case.B_v[0, :128, h * 128:(h + 1) * 128] = torch.eye(128)
    case.zk[0].zero_()
    case.zv[0].zero_()
    case.zk[0][0, :, 0] = torch.as_tensor(a)
    case.zv[0][0, :, :128] = torch.as_tensor(v)
    return case, q, q_pos


@pytest.mark.parametrize("name", ["bf16", "norope"])
def test_weights_keep_float32(name):
    """Sums that cancel show the weights' own error.  Two tokens' weights, exp(-3.425) and exp(-1.978), are
    7.1e-6 above and 6.8e-6 below what two bf16 numbers hold of them, and the values of the 90 tokens of
    the one and the 30 of the other take each other away, so a weight of 16 bits is off by 6.9e-6 Σ p|v|.
    In float32 a score of 5 in base 2 has 5 roundings, 1e-6 of a weight, exp2f 2.4e-7, and the value sums
    of 8 steps of shuffled tokens 2^-23 each of at most the whole: 3e-6 Σ p|v| bounds them together."""
    rng = np.random.default_rng(1)
    kind = rng.permutation(np.array([0] * 8 + [1] * 90 + [2] * 30))
    a = np.array([0.0, -4.84375, -2.796875])[kind]
    x = np.exp(8 * np.array([-4.84375, -2.796875]) / math.sqrt(128.0))
    up = 1 + np.arange(128) / 128
    down = torch.tensor(90 * x[0] * up / (30 * x[1])).to(torch.bfloat16).double().numpy()
    v = np.where(kind[:, None] == 1, up, np.where(kind[:, None] == 2, -down, 0.0))
    case, q, q_pos = one_channel(name, 128, a, v)
    out, _ = run(case, build_pools(case), q, q_pos, [[[[0]]]], 1)
    ref, _, size = S.decode_attention_pages(q[0, 0].double().numpy(), 127, *case.oracle_latents(0), case.positions(0),
                                            case.B_k.double().numpy(), case.B_v.double().numpy(), case.w.group_size,
                                            case.w.rope_base, [[0]], 128, False)
    assert (np.abs(ref / size).min(1) < 1e-4).all()               # the sums do cancel
    assert (np.abs(out[0, 0] - ref) <= HALF_STEP["bf16"] * np.abs(ref) + 3e-6 * size).all()


@pytest.mark.parametrize("name", ["f16_r256", "norope_f16_r256"])
def test_many_small_weights_beside_a_large_one(name):
    """A token that takes nearly all the weight and has no value, beside 999 of weight 2^-25.5 each: below
    the least f16 number, and all of the result.  A score of 25.5 in base 2 has 5 roundings: 5.3e-6."""
    T = 1000
    a = np.full(T, -25.0)
    a[517] = 0.0
    v = np.full((T, 128), 1000.0)
    v[517] = 0.0
    case, q, q_pos = one_channel(name, T, a, v)
    lists = [[[list(range(8))]]]
    out, _ = run(case, build_pools(case), q, q_pos, lists, 8)
    ref, _, size = S.decode_attention_pages(q[0, 0].double().numpy(), T - 1, *case.oracle_latents(0), case.positions(0),
                                            case.B_k.double().numpy(), case.B_v.double().numpy(), case.w.group_size,
                                            case.w.rope_base, lists[0][0], 128, False)
    assert (0.01 < ref).all()
    assert (np.abs(out[0, 0] - ref) <= HALF_STEP["f16"] * np.abs(ref) + 1e-5 * size).all()


@pytest.mark.parametrize("name", ["norope", "norope_f16_r256"])
def test_folded_queries_keep_float32(name):
    """One token a sequence: its log-sum-exp is its score, one product q B_k z of up to 40 on entry 0.
    Scale, query and product are rounded 6 times in float32, 2^-24 of the score each, and to natural
    logarithms twice more; an f16 query keeps 2^-25 of its own, z = 40 times that."""
    w = dataclasses.replace(CASES[name][0], num_heads=4)
    case = make_decode_case(w, [1] * 16)
    q, q_pos = queries(case, 1)
    q.mul_((torch.arange(128) == 40).to(q.dtype)).mul_(4.0)
    case.B_k.zero_()
    for h in range(4):
        case.B_k[0, 0, h * 128 + 40] = 1.0
    for z in case.zk:
        z.zero_()
        z[0, 0, 0] = 40.0
    _, lse = run(case, build_pools(case), q, q_pos, [[[[0]]]] * 16, 1)
    ref = q[:, :, :, 40].double().numpy() * 40.0 / math.sqrt(128.0)
    assert np.abs(ref).max() > 20
    assert (np.abs(lse - ref) <= 8 * 2.0 ** -24 * np.abs(ref) + (40 * 2.0 ** -25 if w.act_dtype == "f16" else 0)).all()


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("name", ["bf16", "f16_r256"])
def test_angles_keep_float32(name, explicit):
    """A sequence's last token, its key one channel of a pair, scores 90 or more for a query one position on
    with entries of one size in both channels, so that an angle off by e changes the score by up to e of it.
    The others score 0: the log-sum-exp is that score, S (cos D + sin D) for an angle D between the two.
    What changes with the position are the angles of query and tile, good to about 2^-24, that of the row
    by the hardware's sine (2^-21.4 at most: a third of it as rms is 1.2e-7) and a dozen roundings of
    2^-24 / sqrt 3 (rms) of at most the score, 1.2e-7: 1.8e-7 of it bounds their spread (the constants'
    roundings shift all)."""
    w = CASES[name][0]
    rng = np.random.default_rng(3)
    lens = rng.integers(1, 3000, 64).tolist()
    case = make_decode_case(w, lens, explicit_positions=explicit)
    q, q_pos = queries(case, 1)
    q.zero_()
    case.B_k.zero_()
    ref = np.empty(w.num_heads)
    for h in range(w.num_heads):
        f = (7 * h + 3) % 64
        q[:, :, h, f], q[:, :, h, f + 64] = 32.0, -32.0
        case.B_k[h // 4, 0, h % 4 * 128 + f] = 1.0
        turn = w.rope_base ** (-f / 64)
        ref[h] = 1024.0 / math.sqrt(128.0) * (math.cos(turn) + math.sin(turn))
    for z, t in zip(case.zk, lens):
        z.zero_()
        z[:, t - 1, 0] = 32.0
    q_pos = np.array([[case.positions(i)[-1] + 1] for i in range(len(lens))], np.int32)
    lists = [[[[(t - 1) // 128]] * w.groups] for t in lens]
    _, lse = run(case, build_pools(case), q, q_pos, lists, 1)
    off = lse[:, 0] / ref - 1
    assert np.abs(off.mean()) < 8 * 2.0 ** -24 and off.std() < 1.8e-7, f"{off.mean():.2e} {off.std():.2e}"


MORE = {
    "int4_f16_norope": (dataclasses.replace(CASES["int4_f16"][0], rope_base=0.0), 2),
    "int4_bf16_norope": (dataclasses.replace(CASES["int4_bf16"][0], rope_base=0.0), 2),
    "norope_d64": (w7b(rope_base=0.0, head_dim=64), 3),
    "norope_d40_three_heads": (dataclasses.replace(w7b(rope_base=0.0, head_dim=40, group_size=3, rank_k=128), num_heads=6), 3),
    "norope_one_head": (dataclasses.replace(w7b(rope_base=0.0, group_size=1, rank_v=256), num_heads=2), 3),
    "eight_heads": (dataclasses.replace(w7b(group_size=8, rank_k=128), num_heads=16), 2),
    "r192_r256": (w7b(rank_k=192, rank_v=256, act_dtype="f16", latent_dtype="f16"), 2),
    "f32_r512": (dataclasses.replace(WORKLOADS["tiny_f32"], rank_k=512, rank_v=512, head_dim=128, page_size=40), 1),
    "f32_r96": (dataclasses.replace(WORKLOADS["tiny_f32"], rank_k=96, rank_v=288), 1),
}


def compare_up(case, out, lse, q, q_pos, lists):
    """compare() for float32, where a query may see so few tokens that an output channel is nearly nothing:
    the up-projection then shows its own roundings.  It runs in 8 chains of r_v / 8 terms and 3 joins on
    sums rounded once: (r_v / 8 + 4)·2^-24 Σ_r |a_r||B_r|, with Σ_r |a_r||B_r| at most the largest token's."""
    w = case.w
    for i, j in np.ndindex(*q_pos.shape):
        zk, zv = case.oracle_latents(i)
        Bk, Bv = case.B_k.double().numpy(), case.B_v.double().numpy()
        ref, rl, size = S.decode_attention_pages(q[i, j].double().numpy(), q_pos[i, j], zk, zv, case.positions(i), Bk, Bv,
                                                 w.group_size, w.rope_base, lists[i][j], w.page_size, q_pos.shape[1] > 1)
        up = np.zeros((w.num_heads, w.head_dim))
        for g in range(w.groups):
            if case.seq_lens[i]:
                up[g * w.group_size:(g + 1) * w.group_size] = (np.abs(zv[g]) @ np.abs(Bv[g])).max(0).reshape(w.group_size, -1)
        off = np.abs(out[i, j] - ref)
        assert (off <= HALF_STEP["f32"] * np.abs(ref) + SUM["f32"] * size + (w.rank_v / 8 + 4) * 2.0 ** -24 * up).all()
        empty = np.isneginf(rl)
        assert (np.isneginf(lse[i, j]) == empty).all()
        np.testing.assert_allclose(lse[i, j][~empty], rl[~empty], rtol=0, atol=LSE["f32"])


@pytest.mark.parametrize("Q", [1, 2])
@pytest.mark.parametrize("name", list(MORE))
def test_more_shapes(name, Q):
    w, kind = MORE[name]
    case = make_decode_case(w, [300, 0, 1, 700])
    assert P.palu_decode_kernel_kind(case.cfg) == kind
    q, q_pos = queries(case, Q)
    lists = pick_lists(case, Q, 4, seed=Q)
    if w.act_dtype == "f32":
        compare_up(case, *run(case, build_pools(case), q, q_pos, lists, 4), q, q_pos, lists)
        return
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 4), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16", "tiny_f32"])
@pytest.mark.parametrize("keep", [200, 5000])
def test_few_pages_in_a_long_list(name, keep):
    case = make_decode_case(CASES[name][0], [300, 0, 900])
    q, q_pos = queries(case, 2)
    lists = pick_lists(case, 2, 3)
    compare(case, *run(case, build_pools(case), q, q_pos, lists, keep), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["bf16", "norope", "int4_f16", "tiny_f32"])
def test_drafts_that_list_the_same_pages(name):
    case = make_decode_case(CASES[name][0], [900, 260])
    q, q_pos = queries(case, 4)
    lists = pick_lists(case, 1, 4)
    lists = [[row[0]] * 4 for row in lists]
    if name == "tiny_f32":
        compare_up(case, *run(case, build_pools(case), q, q_pos, lists, 4), q, q_pos, lists)
        return
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 4), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name,Q,keep,batch", [("bf16", 1, 1, 2100), ("norope", 1, 1, 2100), ("norope", 3, 2, 700),
                                               ("bf16", 2, 1000, 90), ("norope", 2, 1000, 90)])
def test_more_queries_than_one_launch_walks(name, Q, keep, batch):
    """Runs of sequences behind one another: past 2048 queries, or past 128 x 148 x 8 list entries."""
    w = dataclasses.replace(CASES[name][0], num_heads=4, rank_k=64)
    case = make_decode_case(w, [1 + i * 37 % 260 for i in range(batch)])
    q, q_pos = queries(case, Q)
    lists = pick_lists(case, Q, min(keep, 3))
    compare(case, *run(case, build_pools(case), q, q_pos, lists, keep), q, q_pos, lists, uniform(case))


@pytest.mark.parametrize("name", ["tiny_f32", "bf16"])
def test_more_splits_than_a_merge_holds(name):
    case = make_decode_case(CASES[name][0], [700])
    q, q_pos = queries(case, 1)
    lists = [[[[0, 2, 5]] * case.w.groups]]
    compare(case, *run(case, build_pools(case), q, q_pos, lists, 20000, 20000), q, q_pos, lists, uniform(case))
