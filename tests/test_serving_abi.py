"""Host-side refusals of the planning, verification, page-bounds, selection and sparse-decode calls:
statuses of the C ABI and errors of the binding.  CPU only: none of these calls reaches a launch."""
import ctypes

import pytest
import torch

from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200._lib import load

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
A = 1 << 20                                     # a well-aligned address that is never followed


def cfg(**kw):
    base = dict(num_heads=32, head_dim=128, group_size=4, rank_k=256, rank_v=128, page_size=128, rope_base=10000.0,
                act_dtype="bf16", latent_dtype=None)
    return P.make_config(**{**base, **kw})


def call(fn, order, base, **kw):
    v = {**base, **kw}
    return int(getattr(load(), fn)(*[v[k] for k in order]))


PLAN = ["page_size", "batch", "max_pages", "num_pages", "n_rows", "num_new", "seq_lens", "page_table", "free_pages",
        "num_free", "slots", "positions", "row_starts", "taken", "ws", "ws_bytes", "stream"]
PLAN_OK = dict(page_size=128, batch=0, max_pages=4, num_pages=9, n_rows=0, num_new=A, seq_lens=A, page_table=A,
               free_pages=A, num_free=A, slots=A, positions=A, row_starts=A, taken=A, ws=A, ws_bytes=512, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=0), INVALID), (dict(page_size=12), ALIGNMENT), (dict(batch=-1), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(n_rows=-1), INVALID),
    (dict(batch=8193), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=511), WORKSPACE), (dict(ws=A + 64), ALIGNMENT),
    (dict(free_pages=None), INVALID), (dict(num_free=None), INVALID), (dict(batch=2, num_new=None), INVALID),
    (dict(batch=2, seq_lens=None), INVALID), (dict(batch=2, page_table=None), INVALID),
    (dict(n_rows=3, slots=None), INVALID), (dict(n_rows=3, positions=None), INVALID), (dict(seq_lens=A + 2), ALIGNMENT),
])
def test_plan_append(kw, code):
    assert call("palu_plan_append", PLAN, PLAN_OK, **kw) == code


VERIFY = ["dtype", "batch", "D", "V", "p", "p_ld", "q", "q_ld", "tokens_in", "lens", "ua", "us", "tokens", "acc", "back",
          "ws", "ws_bytes", "stream"]
VERIFY_OK = dict(dtype=0, batch=0, D=2, V=100, p=A, p_ld=100, q=A, q_ld=100, tokens_in=A, lens=A, ua=A, us=A, tokens=A,
                 acc=A, back=A, ws=A, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(dtype=3), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(batch=-1), INVALID), (dict(D=-1), INVALID),
    (dict(V=0), INVALID), (dict(D=33), UNSUPPORTED), (dict(batch=8193), UNSUPPORTED), (dict(V=(1 << 28) + 1), UNSUPPORTED),
    (dict(p_ld=99), INVALID), (dict(q_ld=99), INVALID), (dict(q=None, q_ld=0), OK), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=1000), WORKSPACE), (dict(ws=A + 128), ALIGNMENT), (dict(batch=1, p=None), INVALID),
    (dict(batch=1, us=None), INVALID), (dict(batch=1, tokens=None), INVALID), (dict(batch=1, acc=None), INVALID),
    (dict(batch=1, tokens_in=None), INVALID), (dict(batch=1, ua=None), INVALID), (dict(batch=1, p=A + 2), ALIGNMENT),
    (dict(batch=1, q=A + 1), ALIGNMENT), (dict(batch=1, ua=A + 2), ALIGNMENT),
])
def test_verify_drafts(kw, code):
    assert call("palu_verify_drafts", VERIFY, VERIFY_OK, **kw) == code


def test_verify_workspace_grows_with_its_sizes():
    a = P.palu_verify_workspace_size(1, 2, 1000)
    assert P.palu_verify_workspace_size(64, 2, 128000) > a >= 256 + 4 * 8192
    with pytest.raises(P.PaluError):
        P.palu_verify_workspace_size(1, 33, 1000)


BOUNDS = ["cfg", "ranks", "batch", "first", "zk", "zks", "pos", "table", "max_pages", "lens", "num_pages", "Bk", "bounds",
          "ws", "ws_bytes", "stream"]


def bounds_args(**kw):
    return dict(cfg=ctypes.byref(cfg(**kw)), ranks=None, batch=0, first=None, zk=A, zks=None, pos=None, table=A,
                max_pages=4, lens=A, num_pages=9, Bk=A, bounds=A, ws=A, ws_bytes=256, stream=None)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(cfg=None), INVALID), (dict(batch=-1), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=255), WORKSPACE), (dict(ws=A + 16), ALIGNMENT), (dict(batch=1, zk=None), INVALID),
    (dict(batch=1, table=None), INVALID), (dict(batch=1, lens=None), INVALID), (dict(batch=1, Bk=None), INVALID),
    (dict(batch=1, bounds=None), INVALID), (dict(batch=1, num_pages=0), INVALID), (dict(batch=1, zk=A + 8), ALIGNMENT),
    (dict(batch=1, Bk=A + 8), ALIGNMENT), (dict(batch=1, bounds=A + 8), ALIGNMENT),
])
def test_page_bounds(kw, code):
    assert call("palu_page_bounds", BOUNDS, bounds_args(), **kw) == code


@pytest.mark.parametrize("kw", [dict(table=A + 2), dict(lens=A + 2), dict(first=A + 2), dict(pos=A + 1)])
def test_page_bounds_takes_aligned_words(kw):
    assert call("palu_page_bounds", BOUNDS, bounds_args(), batch=1, **kw) == ALIGNMENT


@pytest.mark.parametrize("kw", [dict(table=A + 2), dict(lens=A + 2), dict(q_pos=A + 2), dict(list=A + 2),
                                dict(counts=A + 1), dict(scores=A + 2)])
def test_select_pages_takes_aligned_words(kw):
    assert call("palu_select_pages", SELECT, select_args(), batch=1, **kw) == ALIGNMENT


@pytest.mark.parametrize("kw", [dict(table=A + 2), dict(lens=A + 2), dict(q_pos=A + 2), dict(list=A + 2),
                                dict(counts=A + 1), dict(lse=A + 2), dict(pos=A + 2), dict(out=A + 8)])
def test_decode_attn_pages_takes_aligned_words(kw):
    assert call("palu_decode_attn_pages", ATTEND, attend_args(), batch=1, **kw) == ALIGNMENT


def test_token_counts_past_32_bits():
    wide = 1 << 24                                  # pages of 128 tokens: 2^31 tokens
    assert call("palu_page_bounds", BOUNDS, bounds_args(), max_pages=wide) == UNSUPPORTED
    assert call("palu_page_bounds", BOUNDS, bounds_args(), max_pages=wide - 1) == OK
    assert call("palu_decode_attn_pages", ATTEND, attend_args(), max_pages=wide) == UNSUPPORTED
    assert call("palu_decode_attn_pages", ATTEND, attend_args(), max_pages=wide - 1) == OK
    assert call("palu_decode_attn_pages", ATTEND, attend_args(), keep=wide + 1) == UNSUPPORTED
    big_pages = select_args(page_size=1 << 17)
    assert call("palu_select_pages", SELECT, big_pages, max_pages=1 << 14) == UNSUPPORTED
    assert call("palu_select_pages", SELECT, big_pages, max_pages=(1 << 14) - 1) == OK


def test_page_bounds_configs():
    assert call("palu_page_bounds", BOUNDS, bounds_args(act_dtype="f16", latent_dtype="int4", rank_v=256), batch=1) == INVALID
    assert call("palu_page_bounds", BOUNDS, bounds_args(rank_k=100)) == ALIGNMENT
    bad = (ctypes.c_int32 * 8)(*[256] * 7, 600)
    assert call("palu_page_bounds", BOUNDS, bounds_args(), ranks=bad) == UNSUPPORTED
    assert P.palu_page_bounds_bytes(cfg()) == 2 * 32 * 128 * 2
    assert P.palu_page_bounds_bytes(cfg(act_dtype="f32", rank_k=64, rank_v=64)) == 2 * 32 * 128 * 4


SELECT = ["cfg", "batch", "Q", "q", "q_pos", "bounds", "pos", "table", "max_pages", "lens", "num_pages", "first", "last",
          "keep", "list", "counts", "scores", "ws", "ws_bytes", "stream"]


def select_args(**kw):
    return dict(cfg=ctypes.byref(cfg(**kw)), batch=0, Q=1, q=A, q_pos=A, bounds=A, pos=None, table=A, max_pages=4, lens=A,
                num_pages=9, first=1, last=2, keep=4, list=A, counts=A, scores=None, ws=A, ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(cfg=None), INVALID), (dict(batch=-1), INVALID), (dict(Q=0), INVALID), (dict(Q=17), INVALID),
    (dict(max_pages=0), INVALID), (dict(num_pages=-1), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(keep=0, first=0, last=0), INVALID), (dict(keep=2), INVALID), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID),
    (dict(batch=8193), UNSUPPORTED), (dict(max_pages=32769), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(batch=1, ws_bytes=262144), WORKSPACE), (dict(ws=A + 32), ALIGNMENT), (dict(batch=1, q=None), INVALID),
    (dict(batch=1, q_pos=None), INVALID), (dict(batch=1, bounds=None), INVALID), (dict(batch=1, table=None), INVALID),
    (dict(batch=1, lens=None), INVALID), (dict(batch=1, list=None), INVALID), (dict(batch=1, counts=None), INVALID),
    (dict(batch=1, num_pages=0), INVALID), (dict(batch=1, q=A + 4), ALIGNMENT), (dict(batch=1, bounds=A + 4), ALIGNMENT),
])
def test_select_pages(kw, code):
    assert call("palu_select_pages", SELECT, select_args(), **kw) == code


def test_select_group_width():
    wide = select_args(num_heads=128, group_size=128, rank_k=64, rank_v=64)
    assert call("palu_select_pages", SELECT, wide) == UNSUPPORTED


ATTEND = ["cfg", "rk", "rv", "batch", "Q", "q", "q_pos", "zk", "zv", "zks", "zvs", "pos", "table", "max_pages", "lens", "list",
          "counts", "keep", "num_pages", "Bk", "Bv", "out", "lse", "ws", "ws_bytes", "splits", "stream"]


def attend_args(**kw):
    return dict(cfg=ctypes.byref(cfg(**kw)), rk=None, rv=None, batch=0, Q=1, q=A, q_pos=A, zk=A, zv=A, zks=None, zvs=None,
                pos=None, table=A, max_pages=4, lens=A, list=A, counts=A, keep=3, num_pages=9, Bk=A, Bv=A, out=A, lse=None,
                ws=A, ws_bytes=1 << 24, splits=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(cfg=None), INVALID), (dict(batch=-1), INVALID), (dict(Q=0), INVALID), (dict(Q=17), INVALID),
    (dict(keep=0), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=-1), INVALID), (dict(splits=-1), INVALID),
    (dict(splits=4), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(batch=8192, Q=9), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(batch=1, ws_bytes=256), WORKSPACE), (dict(ws=A + 64), ALIGNMENT),
    *[(dict(batch=1, **{k: None}), INVALID) for k in ("q", "q_pos", "zk", "zv", "table", "lens", "list", "counts", "Bk",
                                                      "Bv", "out")],
    (dict(batch=1, num_pages=0), INVALID), (dict(batch=1, q=A + 8), ALIGNMENT), (dict(batch=1, zv=A + 8), ALIGNMENT),
])
def test_decode_attn_pages(kw, code):
    assert call("palu_decode_attn_pages", ATTEND, attend_args(), **kw) == code


def test_decode_pages_workspace_size():
    lib, n = load(), ctypes.c_size_t()
    args = lambda b=4, Q=1, keep=8, s=0: (ctypes.byref(cfg()), None, None, b, Q, keep, s, ctypes.byref(n))
    assert lib.palu_decode_pages_workspace_size(*args()) == OK and n.value >= 256 + 4 * 32 * (128 + 8) * 4
    small = n.value
    assert lib.palu_decode_pages_workspace_size(*args(b=64)) == OK and n.value > small
    for bad in (dict(b=-1), dict(Q=0), dict(Q=17), dict(keep=0), dict(s=-1), dict(s=9)):
        assert lib.palu_decode_pages_workspace_size(*args(**bad)) == INVALID
    assert lib.palu_decode_pages_workspace_size(*args(b=65536)) == UNSUPPORTED
    # a layer is as large as its largest set, and one launch's worth of a large batch bounds it
    assert P.palu_decode_pages_workspace_size(cfg(), 60000, 1, 4096) < 1 << 30


# ------------------------------------------------------------------ the binding
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
ws = lambda n=4096: torch.zeros(n, dtype=torch.uint8)


def test_binding_refuses_shapes_types_and_host_memory():
    good = dict(num_new=i32(4), seq_lens=i32(4), page_table=i32(4, 3), free_pages=i32(9), num_free=i32(1),
                slot_mapping=i32(7), positions=i32(7), row_starts=i32(5), taken=i32(4), workspace=ws())
    for k, bad in (("num_new", i32(5)), ("seq_lens", i32(4).long()), ("page_table", i32(3, 4).t()), ("num_free", i32(2)),
                   ("positions", i32(6)), ("row_starts", i32(4)), ("taken", i32(3)), ("slot_mapping", i32(7, 1))):
        with pytest.raises(ValueError, match=k if k != "slot_mapping" else "slot_mapping|positions"):
            P.palu_plan_append(128, **{**good, k: bad})
    with pytest.raises(ValueError, match="CUDA"):
        P.palu_plan_append(128, **good)
    with pytest.raises(TypeError, match="workspace"):
        P.palu_plan_append(128, **{**good, "workspace": None})
    with pytest.raises(TypeError, match="num_new"):
        P.palu_plan_append(128, **{**good, "num_new": [1, 2, 3, 4]})


def test_binding_takes_evenly_spaced_rows_only():
    p = torch.zeros((3, 2, 16))
    rest = (torch.zeros((3, 1), dtype=torch.int32), None, torch.zeros((3, 1)), torch.zeros(3), i32(3, 2), i32(3), i32(3), ws())
    with pytest.raises(ValueError, match="CUDA"):
        P.palu_verify_drafts(p[..., :11], None, *rest)                     # a slice of padded rows will do
    with pytest.raises(ValueError, match="evenly spaced"):
        P.palu_verify_drafts(p[..., ::2], None, *rest)
    with pytest.raises(ValueError, match="evenly spaced"):
        P.palu_verify_drafts(torch.zeros((3, 3, 16))[:, :2], None, *rest)  # a gap after every two rows
    with pytest.raises(ValueError, match="float32, float16 or bfloat16"):
        P.palu_verify_drafts(p.double(), None, *rest)
    with pytest.raises(ValueError, match="draft_probs"):
        P.palu_verify_drafts(p, torch.zeros((3, 1, 16), dtype=torch.bfloat16), *rest)


def test_binding_checks_pool_sizes():
    c = cfg(num_heads=4)
    pages, bf = 2, torch.bfloat16
    pool = lambda n: torch.zeros(n, dtype=torch.uint8)
    zk, bounds, Bk = pool(2 * 128 * 512), torch.zeros(2 * 2 * 512, dtype=bf), torch.zeros((256, 512), dtype=bf)
    with pytest.raises(ValueError, match="zk_pool holds fewer"):
        P.palu_page_bounds(c, None, zk[1:], None, None, i32(1, 2), i32(1), pages, Bk, bounds, ws())
    with pytest.raises(ValueError, match="bounds holds fewer"):
        P.palu_page_bounds(c, None, zk, None, None, i32(1, 2), i32(1), pages, Bk, bounds[1:], ws())
    with pytest.raises(ValueError, match="B_k must hold"):
        P.palu_page_bounds(c, None, None, None, None, i32(0, 2), i32(0), pages, Bk[:128], bounds, ws())
    q = torch.zeros((1, 1, 4, 128), dtype=bf)
    with pytest.raises(ValueError, match="page_list"):
        P.palu_select_pages(c, q, i32(1, 1), bounds, None, i32(1, 2), i32(1), pages, 0, 0, i32(1, 2, 1, 4), i32(1, 1, 1),
                            None, ws())
    with pytest.raises(ValueError, match="zv_pool holds fewer"):
        P.palu_decode_attn_pages(c, q, i32(1, 1), None, zk[:100], None, None, None, i32(1, 2), i32(1), i32(1, 1, 1, 4),
                                 i32(1, 1, 1), pages, Bk, Bk[:128], q, None, ws())


def test_binding_checks_the_number_of_ranks():
    c = cfg()
    with pytest.raises(ValueError, match="8 head groups"):
        P.palu_page_bounds(c, None, None, None, None, i32(0, 2), i32(0), 1, ws(), ws(), ws(), ranks_k=[256] * 7)
    with pytest.raises(ValueError, match="8 head groups"):
        P.palu_decode_pages_workspace_size(c, 1, 1, 4, ranks_k=[256] * 8, ranks_v=[128] * 9)
    with pytest.raises(ValueError, match="together"):
        P.palu_decode_pages_workspace_size(c, 1, 1, 4, ranks_k=[256] * 8)
    empty = cfg()
    empty.group_size = 0
    with pytest.raises(P.PaluError):
        P.palu_decode_pages_workspace_size(empty, 1, 1, 4)


def test_binding_takes_int32_positions_only():
    c = cfg(num_heads=4)
    bf = torch.bfloat16
    zk, bounds, Bk = ws(128 * 512), torch.zeros(2 * 512, dtype=bf), torch.zeros((256, 512), dtype=bf)
    q, pos = torch.zeros((1, 1, 4, 128), dtype=bf), torch.zeros(128, dtype=torch.int64)
    with pytest.raises(ValueError, match="pos_pool"):
        P.palu_page_bounds(c, None, zk, None, pos, i32(1, 2), i32(1), 1, Bk, bounds, ws())
    with pytest.raises(ValueError, match="pos_pool"):
        P.palu_decode_attn_pages(c, q, i32(1, 1), zk, zk, None, None, pos, i32(1, 2), i32(1), i32(1, 1, 1, 4),
                                 i32(1, 1, 1), 1, Bk, Bk[:128], q, None, ws())
    with pytest.raises(ValueError, match="pos_pool"):
        P.palu_select_pages(c, q, i32(1, 1), bounds, pos, i32(1, 2), i32(1), 1, 0, 0, i32(1, 1, 1, 4), i32(1, 1, 1), None,
                            ws())
