"""palu_page_bounds on the GPU against the CPU oracle.

Error bounds, per key entry: the float32 (tensor-core) product of r terms is off by at most r·2^-23
Σ|z||B| (2^-24 per rounding, doubled for truncating adders), a rotation mixes two entries and its
angles are exact to 2^-20 (the hardware sine at explicit positions), and the outward rounding moves a
bound away by less than one step, 2^-7 (bf16), 2^-10 (f16) of its size.
"""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from palu_testlib import build_pools, build_ranked_pools, make_decode_case, make_ranked_case
from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200.synth import TORCH_DTYPE, WORKLOADS

pytestmark = pytest.mark.gpu
STEP = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10, "f32": 0.0}
FILL = 7.0


def run(cfg, case, pools, B_k, first=None, ranks_k=None, bounds=None):
    w = case.w
    G, W = w.groups, w.width
    if bounds is None:
        bounds = torch.full((case.num_pages, G, 2, W), FILL, dtype=TORCH_DTYPE[w.act_dtype], device="cuda")
    b, mp = case.page_table.shape
    ws = torch.zeros(P.palu_page_bounds_workspace_size(cfg, b, mp), dtype=torch.uint8, device="cuda")
    P.palu_page_bounds(cfg, None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda"),
                       pools["zk"], pools["zks"], pools["pos"], torch.from_numpy(case.page_table).cuda(),
                       torch.tensor(case.seq_lens, dtype=torch.int32, device="cuda"), case.num_pages, B_k.cuda(),
                       bounds, ws, ranks_k=ranks_k)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == 0
    return bounds


def check(case, bounds, keys, first=None):
    """keys(i) -> per group (z_k [T, r], B_k [r, W]) in float64."""
    w = case.w
    got = bounds.double().cpu().numpy()
    touched = set()
    for i, T in enumerate(case.seq_lens):
        pos = case.positions(i)
        for g, (z, B) in enumerate(keys(i)):
            if T == 0:
                continue
            lo, hi = S.page_bounds(z, pos, B, w.head_dim, w.rope_base, w.page_size)
            slack = 1.5 * np.max(np.abs(z) @ np.abs(B)) * (z.shape[1] * 2.0 ** -23 + 2.0 ** -19)
            for lp in range(len(lo)):
                if first is not None and (lp + 1) * w.page_size <= first[i]:
                    continue
                touched.add(int(case.page_table[i, lp]))
                a, b = got[case.page_table[i, lp], g]
                assert (a <= lo[lp] + slack).all() and (b >= hi[lp] - slack).all(), f"seq {i} page {lp} group {g}"
                assert (a >= lo[lp] - slack - STEP[w.act_dtype] * np.abs(lo[lp])).all(), f"seq {i} page {lp} low"
                assert (b <= hi[lp] + slack + STEP[w.act_dtype] * np.abs(hi[lp])).all(), f"seq {i} page {lp} high"
    for pg in set(range(case.num_pages)) - touched:
        assert (got[pg] == FILL).all(), f"page {pg} written"


def uniform(case):
    def keys(i):
        zk, _ = case.oracle_latents(i)
        B = case.B_k.double().numpy()
        return [(zk[g], B[g]) for g in range(case.w.groups)]
    return keys


def w7b(**kw):
    return dataclasses.replace(WORKLOADS["7b_bf16_r256v128_b1_t4k"], num_heads=8, **kw)


CASES = {
    "bf16": w7b(),
    "f16_r64": w7b(act_dtype="f16", latent_dtype="f16", rank_k=64),
    "bf16_two_heads_r192": w7b(group_size=2, rank_k=192),
    "norope": w7b(rope_base=0.0),
    "int4_f16": dataclasses.replace(WORKLOADS["7b_int4_r256_b8_t32k"], num_heads=8),
    "int4_bf16": dataclasses.replace(WORKLOADS["7b_int4_r256_b8_t32k"], num_heads=8, act_dtype="bf16"),
    "tiny_f32": WORKLOADS["tiny_f32"],
    "f32_norope": dataclasses.replace(WORKLOADS["tiny_f32"], rope_base=0.0, page_size=16),
    "odd_heads": dataclasses.replace(WORKLOADS["tiny_f32"], num_heads=6, group_size=3, head_dim=40, act_dtype="bf16",
                                     latent_dtype="bf16", page_size=24),
    "int4_small": dataclasses.replace(WORKLOADS["tiny_f32"], num_heads=4, group_size=2, rank_k=256, rank_v=256,
                                      act_dtype="f16", latent_dtype="int4", page_size=64),
}


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_bounds(name, explicit):
    case = make_decode_case(CASES[name], [300, 0, 1, 128, 515], explicit_positions=explicit)
    check(case, run(case.cfg, case, build_pools(case), case.B_k), uniform(case))


@pytest.mark.parametrize("name", ["bf16", "int4_f16", "tiny_f32"])
def test_only_pages_from_the_first_token_on(name):
    case = make_decode_case(CASES[name], [300, 0, 1, 256, 700])
    first = [299, 0, 0, 256, 130]
    check(case, run(case.cfg, case, build_pools(case), case.B_k, first), uniform(case), first)


def test_many_sequences_and_long_ones():
    case = make_decode_case(w7b(), [5 + 37 * i for i in range(40)])
    check(case, run(case.cfg, case, build_pools(case), case.B_k), uniform(case))
    case = make_decode_case(w7b(), [9000])
    check(case, run(case.cfg, case, build_pools(case), case.B_k), uniform(case))


def test_more_sequences_than_one_launch_enumerates():
    case = make_decode_case(dataclasses.replace(w7b(), num_heads=4, rank_k=64, rank_v=128),
                            [1 + (i % 3) for i in range(2100)])
    check(case, run(case.cfg, case, build_pools(case), case.B_k), uniform(case))


@pytest.mark.parametrize("ranks_k", [[64, 256], [192, 128]])
def test_ranks_per_group(ranks_k):
    case = make_ranked_case(w7b(), ranks_k, [128, 128], [300, 129])
    pools = build_ranked_pools(case)

    def keys(i):
        zk, _, Bk, _ = case.oracle_inputs(i)
        return list(zip(zk, Bk))

    check(case, run(case.cfg, case, pools, case.B_k, ranks_k=ranks_k), keys)


@pytest.mark.parametrize("name", ["bf16", "tiny_f32"])
def test_rows_behind_the_last_token_do_not_count(name):
    """NaN and infinities in the unused rows of a partial page change nothing."""
    case = make_decode_case(CASES[name], [133, 7])
    pools = build_pools(case)
    ref = run(case.cfg, case, pools, case.B_k)
    w = case.w
    T = TORCH_DTYPE[w.latent_dtype]
    row = w.rank_k * T.itemsize
    raw = pools["zk"].view(case.num_pages, w.groups, row // 128, w.page_size, 128)
    for i, t in enumerate(case.seq_lens):
        page = int(case.page_table[i, t // w.page_size])
        junk = raw[page, :, :, t % w.page_size:].contiguous().view(T)
        junk[..., 0::2], junk[..., 1::2] = float("nan"), float("inf")
        raw[page, :, :, t % w.page_size:] = junk.view(torch.uint8)
    assert torch.equal(run(case.cfg, case, pools, case.B_k).view(torch.uint8), ref.view(torch.uint8))


def test_half_precision_overflow_rounds_outwards():
    """Keys beyond the largest half: the upper bound is infinite, the lower one finite where it can be."""
    case = make_decode_case(CASES["f16_r64"], [128])
    case.B_k.mul_(30000.0)
    got = run(case.cfg, case, build_pools(case), case.B_k)[case.page_table[0, 0]].float()
    assert torch.isinf(got[:, 1]).any() and not torch.isnan(got).any()
    assert (got[:, 0] <= got[:, 1]).all()


def test_a_bad_page_is_reported_and_skipped():
    case = make_decode_case(CASES["bf16"], [300])
    case.page_table[0, 1] = case.num_pages + 5
    b = torch.full((case.num_pages, 2, 2, 512), FILL, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(P.palu_page_bounds_workspace_size(case.cfg, 1, 3), dtype=torch.uint8, device="cuda")
    pools = dict(build_pools(make_decode_case(CASES["bf16"], [300])))
    P.palu_page_bounds(case.cfg, None, pools["zk"], None, None, torch.from_numpy(case.page_table).cuda(),
                       torch.tensor([300], dtype=torch.int32, device="cuda"), case.num_pages, case.B_k.cuda(), b, ws)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == 7
    assert sum(bool((b[p] != FILL).any()) for p in range(case.num_pages)) == 2


def test_timeout_reports_and_recovers():
    case = make_decode_case(CASES["bf16"], [300])
    pools = build_pools(case)
    b = torch.zeros((case.num_pages, 2, 2, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(P.palu_page_bounds_workspace_size(case.cfg, 1, 3), dtype=torch.uint8, device="cuda")
    P.palu_debug_timeout_test(1 << 20, stall=True)
    try:
        P.palu_page_bounds(case.cfg, None, pools["zk"], None, None, torch.from_numpy(case.page_table).cuda(),
                           torch.tensor([300], dtype=torch.int32, device="cuda"), case.num_pages, case.B_k.cuda(), b, ws)
    finally:
        P.palu_debug_timeout_test()
    st, detail = P.palu_get_device_status(ws)
    assert st == 6 and detail < 90000
    check(case, run(case.cfg, case, pools, case.B_k), uniform(case))


@pytest.mark.parametrize("name", ["bf16", "f16_r64", "tiny_f32"])
def test_bounds_enclose_entries_that_cancel_at_explicit_positions(name):
    """One token a page, its key 1 in both channels of a pair, at positions where the rotated entry cos - sin
    nearly vanishes: its outward rounding hides nothing then.  Sine and cosine are good to 2^-23.5 each, the
    products and the difference of two near numbers are exact."""
    w = CASES[name]
    half = w.head_dim // 2
    pick = []
    for f in (1, 5, 9, 13):
        p = np.arange(1, 2 ** 22, dtype=np.int64)
        x = np.abs(np.remainder(p * w.rope_base ** (-f / half), 2 * np.pi) - np.pi / 4)
        pick += [(f, int(i)) for i in p[np.argsort(x)[:60]]]
    case = make_decode_case(w, [1] * len(pick), explicit_positions=True)
    case.pos = [np.array([p], np.int32) for _, p in pick]
    case.B_k.zero_()
    for i, f in enumerate((1, 5, 9, 13)):
        case.B_k[:, i, f] = case.B_k[:, i, f + half] = 1.0
    for z, (f, _) in zip(case.zk, pick):
        z.zero_()
        z[:, 0, (f - 1) // 4] = 1.0
    got = run(case.cfg, case, build_pools(case), case.B_k).double().cpu().numpy()
    for i, (f, p) in enumerate(pick):
        k = S.page_keys(np.ones((1, 1)), [p], np.eye(w.head_dim)[[f]] + np.eye(w.head_dim)[[f + half]], w.head_dim, w.rope_base)[0]
        assert abs(k[f]) < 1e-4
        lo, hi = got[case.page_table[i, 0], 0][:, [f, f + half]]
        assert (lo <= k[[f, f + half]] + 2 * 2.0 ** -23.5).all() and (hi >= k[[f, f + half]] - 2 * 2.0 ** -23.5).all(), f"{f} {p}"


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("name", ["int4_f16", "int4_bf16", "bf16"])
def test_bounds_without_rope(name, explicit):
    case = make_decode_case(dataclasses.replace(CASES[name], rope_base=0.0), [300, 0, 1, 515], explicit_positions=explicit)
    check(case, run(case.cfg, case, build_pools(case), case.B_k), uniform(case))


@pytest.mark.parametrize("ranks_k", [[64, 512], [320, 256]])
def test_a_key_rank_past_256(ranks_k):
    """The whole layer takes the CUDA-core kernel."""
    case = make_ranked_case(w7b(), ranks_k, [128, 128], [140, 9])

    def keys(i):
        zk, _, Bk, _ = case.oracle_inputs(i)
        return list(zip(zk, Bk))

    check(case, run(case.cfg, case, build_ranked_pools(case), case.B_k, ranks_k=ranks_k), keys)


def test_a_wide_table_is_counted_in_several_launches():
    """160 sequences of up to 2^24 - 1 pages: together more pages than 32 bits count, of which a few are rebuilt."""
    w = dataclasses.replace(w7b(), num_heads=4, rank_k=64, rank_v=128)
    wide = 2 ** 24 - 1
    case = make_decode_case(w, [130] * 160)
    narrow = torch.from_numpy(case.page_table).cuda()
    table = torch.full((160, wide), -1, dtype=torch.int32, device="cuda")
    table[:, :2] = narrow
    launches = P.palu_kernel_launches()
    bounds = torch.full((case.num_pages, 1, 2, 512), FILL, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(P.palu_page_bounds_workspace_size(case.cfg, 160, wide), dtype=torch.uint8, device="cuda")
    pools = build_pools(case)
    P.palu_page_bounds(case.cfg, None, pools["zk"], None, None, table, torch.full((160,), 130, dtype=torch.int32, device="cuda"),
                       case.num_pages, case.B_k.cuda(), bounds, ws)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == 0 and P.palu_kernel_launches() == launches + 2
    check(case, bounds, uniform(case))
