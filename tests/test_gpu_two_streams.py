"""Calls that overlap on the GPU, each on a stream and a workspace of its own: every result is to the bit
what the call gives alone."""
import numpy as np
import pytest
import torch

import test_gpu_decode_pages as D
import test_gpu_select_pages as L
import test_gpu_verify_drafts as V
from palu_testlib import build_pools, make_decode_case
from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200.synth import TORCH_DTYPE

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def attend(name, Q, lens, keep, seed):
    case = make_decode_case(D.CASES[name][0], lens, seed=seed)
    w, b = case.w, len(lens)
    q, q_pos = D.queries(case, Q, seed)
    lists = D.pick_lists(case, Q, keep, seed)
    flat, counts = np.full((b, Q, w.groups, keep), -1, np.int32), np.zeros((b, Q, w.groups), np.int32)
    for i, j, g in np.ndindex(b, Q, w.groups):
        flat[i, j, g, :len(lists[i][j][g])] = lists[i][j][g]
        counts[i, j, g] = len(lists[i][j][g])
    pools = build_pools(case)
    out = torch.zeros((b, Q, w.num_heads, w.head_dim), dtype=TORCH_DTYPE[w.act_dtype], device="cuda")
    lse = torch.zeros((b, Q, w.num_heads), device="cuda")
    ws = torch.zeros(P.palu_decode_pages_workspace_size(case.cfg, b, Q, keep), dtype=torch.uint8, device="cuda")
    args = (q.cuda(), dev(q_pos), pools["zk"], pools["zv"], pools["zks"], pools["zvs"], pools["pos"], dev(case.page_table),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), dev(flat), dev(counts), case.num_pages, case.B_k.cuda(),
            case.B_v.cuda(), out, lse, ws)
    return lambda: P.palu_decode_attn_pages(case.cfg, *args), (out, lse), ws


def bounds(name, lens, seed):
    case = make_decode_case(D.CASES[name][0], lens, seed=seed)
    pools, b = build_pools(case), len(lens)
    out = torch.zeros((case.num_pages, case.w.groups, 2, case.w.width), dtype=TORCH_DTYPE[case.w.act_dtype], device="cuda")
    ws = torch.zeros(P.palu_page_bounds_workspace_size(case.cfg, b, case.page_table.shape[1]), dtype=torch.uint8, device="cuda")
    args = (None, pools["zk"], pools["zks"], pools["pos"], dev(case.page_table),
            torch.tensor(lens, dtype=torch.int32, device="cuda"), case.num_pages, case.B_k.cuda(), out, ws)
    return lambda: P.palu_page_bounds(case.cfg, *args), (out,), ws


def select(seed):
    c = L.make(L.SHAPES["7b_bf16"], [40000, 9000, 300], Q=2, seed=seed)
    cfg, w = L.cfg_of(c["w"]), c["w"]
    lists = torch.zeros((3, 2, w.groups, 9), dtype=torch.int32, device="cuda")
    counts, scores = torch.zeros((3, 2, w.groups), dtype=torch.int32, device="cuda"), torch.zeros(lists.shape, device="cuda")
    ws = torch.zeros(P.palu_select_workspace_size(cfg, 3, 2, c["table"].shape[1]), dtype=torch.uint8, device="cuda")
    args = (c["q"].cuda(), c["q_pos"].cuda(), c["bounds"].cuda(), None, c["table"].cuda(),
            torch.tensor(c["lens"], dtype=torch.int32, device="cuda"), c["pages"], 1, 2, lists, counts, scores, ws)
    return lambda: P.palu_select_pages(cfg, *args), (lists, counts, scores), ws


def verify(seed):
    c = V.make(9, 3, 30011, "bf16", seed=seed)
    out, acc = torch.zeros((9, 4), dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    ws = torch.zeros(P.palu_verify_workspace_size(9, 3, 30011), dtype=torch.uint8, device="cuda")
    args = [c[k].cuda() for k in ("target", "draft", "tokens", "lens", "ua", "us")]
    return lambda: P.palu_verify_drafts(*args, out, acc, None, ws), (out, acc), ws


@pytest.mark.parametrize("pair", ["bf16+bf16", "bf16+norope", "norope+norope", "int4+bf16", "bounds+bf16", "bounds+bounds",
                                  "select+norope", "verify+select", "float32+float32"])
def test_two_streams(pair):
    made = {"bf16": lambda s: attend("bf16", 2, [2000, 0, 900, 1], 9, s), "norope": lambda s: attend("norope", 2, [1500, 70], 7, s),
            "int4": lambda s: attend("int4_f16", 1, [1800, 333], 8, s), "float32": lambda s: attend("tiny_f32", 1, [600], 3, s),
            "bounds": lambda s: bounds("bf16", [3000, 129], s), "select": select, "verify": verify}
    calls = [made[name](seed) for seed, name in enumerate(pair.split("+"), 1)]
    alone = []
    for call, out, _ in calls:
        call()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(30):
        for _, out, _ in calls:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for n in range(6):                       # enough to keep both streams busy at once
            for (call, _, _), stream in zip(calls, streams):
                with torch.cuda.stream(stream):
                    call()
        torch.cuda.synchronize()
        for (_, out, ws), want in zip(calls, alone):
            assert P.palu_get_device_status(ws)[0] == 0
            for x, y in zip(out, want):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
