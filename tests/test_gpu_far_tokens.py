"""Sequences whose token count plus a page passes 2^31: every page of the table is the one real page."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200.synth import normal_tensor

pytestmark = pytest.mark.gpu
# (page size, pages): the product is below 2^31, a page more is not
SIZES = [(65544, 32764), (1000000, 2147)]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@dataclasses.dataclass
class Far:
    """A float32 layer of one head of 8 at rank 32 whose last page holds `left` of its tokens."""
    page: int
    wide: int
    left: int

    def __post_init__(self):
        self.tokens = (self.wide - 1) * self.page + self.left
        assert self.tokens < 2 ** 31 <= self.tokens + self.page
        self.cfg = P.make_config(1, 8, 1, 32, 32, self.page, 10000.0, "f32")
        self.z = normal_tensor(1, "z", (self.left, 32), "f32")
        self.B = normal_tensor(1, "B", (32, 8), "f32", 1 / math.sqrt(32))
        self.q = normal_tensor(1, "q", (1, 1, 1, 8), "f32")
        pool = torch.zeros((self.page, 32))              # 128 bytes a token, its 16-byte units exchanged by t mod 8
        t = torch.arange(self.left)
        unit = torch.arange(8)[None, :] ^ (t[:, None] % 8)
        pool[:self.left].view(-1, 8, 4).scatter_(1, unit[:, :, None].expand(-1, -1, 4), self.z.view(-1, 8, 4))
        self.pool = pool.cuda().view(torch.uint8).view(-1)
        self.table, self.lens = torch.zeros((1, self.wide), dtype=torch.int32, device="cuda"), i32([self.tokens])

    def last(self):
        """Positions of the last page's tokens."""
        return np.arange(self.left) + (self.wide - 1) * self.page


@pytest.mark.parametrize("page,wide", SIZES)
def test_bounds(page, wide):
    f = Far(page, wide, page - 5)
    bounds = torch.full((1, 1, 2, 8), 7.0, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    P.palu_page_bounds(f.cfg, i32([f.tokens - 1]), f.pool, None, None, f.table, f.lens, 1, f.B.cuda(), bounds, ws)
    assert P.palu_get_device_status(ws)[0] == 0
    k = S.page_keys(f.z.double().numpy(), f.last(), f.B.double().numpy(), 8, 10000.0)
    got = bounds.double().cpu().numpy()[0, 0]
    # 33 roundings of 2^-24 of |z||B| <= 20, angles good to 2^-23
    assert np.abs(got[0] - k.min(0)).max() < 5e-5 and np.abs(got[1] - k.max(0)).max() < 5e-5


@pytest.mark.parametrize("page,wide", SIZES)
def test_attend(page, wide):
    f = Far(page, wide, page - 5)
    f.left = 200                                         # (the oracle's part: the first tokens of the last page)
    out, lse = torch.full((1, 1, 1, 8), 7.0, device="cuda"), torch.full((1, 1, 1), 7.0, device="cuda")
    ws = torch.zeros(P.palu_decode_pages_workspace_size(f.cfg, 1, 2, 1), dtype=torch.uint8, device="cuda")
    seen = (wide - 1) * page + 199                       # the first of two queries sees 200 tokens of the page
    q = f.q.expand(1, 2, 1, 8).contiguous().cuda()
    out, lse = out.repeat(1, 2, 1, 1), lse.repeat(1, 2, 1)
    P.palu_decode_attn_pages(f.cfg, q, i32([[seen, f.tokens - 1]]), f.pool, f.pool, None, None, None, f.table, f.lens,
                             i32([[[[wide - 1]], [[wide - 1]]]]), i32([[[1], [1]]]), 1, f.B.cuda(), f.B.cuda(), out, lse, ws)
    assert P.palu_get_device_status(ws)[0] == 0
    z, B = f.z[:200].double().numpy(), f.B.double().numpy()
    ref, rl, size = S.decode_attention_pages(f.q[0, 0].double().numpy(), seen, z[None], z[None], f.last(), B[None], B[None],
                                             1, 10000.0, [[0]], 200, False)
    # as the other float32 cases: a score's error 1e-5, a weight's with it, and the up-projection's
    # (32 / 8 + 4)·2^-24 of Σ |a||B| <= 6
    assert np.abs(lse[0, 0].double().cpu().numpy() - rl).max() < 1e-5
    assert (np.abs(out[0, 0].double().cpu().numpy() - ref) <= 2e-5 * size + 3e-6).all()


@pytest.mark.parametrize("page,wide", SIZES)
def test_select(page, wide):
    f = Far(page, wide, page - 5)
    bounds = torch.ones((1, 1, 2, 8), device="cuda")
    lists, counts = torch.full((1, 1, 1, 4), 99, dtype=torch.int32, device="cuda"), i32([[[99]]])
    ws = torch.zeros(P.palu_select_workspace_size(f.cfg, 1, 1, wide), dtype=torch.uint8, device="cuda")
    P.palu_select_pages(f.cfg, f.q.cuda(), i32([[f.tokens - 1]]), bounds, None, f.table, f.lens, 1, 0, 1, lists, counts, None,
                        ws)
    assert P.palu_get_device_status(ws)[0] == 0
    assert lists.tolist() == [[[[0, 1, 2, wide - 1]]]] and counts.tolist() == [[[4]]]      # equal scores: the lowest


@pytest.mark.parametrize("page,wide", SIZES)
def test_plan(page, wide):
    lens, table = i32([(wide - 1) * page + page - 9]), torch.zeros((1, wide), dtype=torch.int32, device="cuda")
    slots, positions, starts, taken = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (9, 9, 2, 1))
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    P.palu_plan_append(page, i32([9]), lens, table, i32([0]), i32([0]), slots, positions, starts, taken, ws)
    assert P.palu_get_device_status(ws)[0] == 0
    assert slots.tolist() == list(range(page - 9, page)) and taken.tolist() == [9] and lens.tolist() == [wide * page]
    assert positions.tolist() == list(range(wide * page - 9, wide * page))
