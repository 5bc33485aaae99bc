"""palu_plan_append on the GPU against the CPU oracle: every output is a whole number and equal."""
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from rank_kv_cache_palu_b200 import api as P

pytestmark = pytest.mark.gpu


def make_state(rng, batch, page, wide, num_pages, fill=0.5):
    lens = [rng.randint(0, int(fill * wide * page)) for _ in range(batch)]
    order = rng.sample(range(num_pages), num_pages)
    table = [[-1] * wide for _ in range(batch)]
    for b, t in enumerate(lens):
        for lp in range(-(-t // page)):
            table[b][lp] = order.pop()
    return lens, table, order + [-1] * (num_pages - len(order)), len(order)


class Plan:
    """The state of a server on the GPU, and its planning calls."""

    def __init__(self, page, lens, table, stack, free, n_rows):
        i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        self.page, self.batch = page, len(lens)
        self.lens, self.table, self.stack, self.free = i(lens), i(table), i(stack), i([free])
        self.slots, self.positions = i([77] * n_rows), i([77] * n_rows)
        self.starts, self.taken = i([77] * (self.batch + 1)), i([77] * self.batch)
        self.ws = torch.zeros(P.palu_plan_workspace_size(self.batch), dtype=torch.uint8, device="cuda")

    def call(self, new, starts=True, **kw):
        P.palu_plan_append(self.page, new, self.lens, self.table, self.stack, self.free, self.slots, self.positions,
                           self.starts if starts else None, self.taken if starts else None, self.ws, **kw)

    def check(self, ref, free=None):
        torch.cuda.synchronize()
        got = dict(seq_lens=self.lens, page_table=self.table, free_pages=self.stack, slot_mapping=self.slots,
                   positions=self.positions, row_starts=self.starts, taken=self.taken)
        for k, v in got.items():
            np.testing.assert_array_equal(v.cpu().numpy(), np.array(ref[k]).reshape(v.shape), err_msg=k)
        assert int(self.free) == ref["num_free"]
        assert P.palu_get_device_status(self.ws)[0] == (7 if ref["fault"] else 0)
        assert int(self.ws[256:].sum()) == 0              # counters back at zero


def run_case(rng, batch, page, wide, num_pages, new, n_rows, free=None, fill=0.5):
    lens, table, stack, had = make_state(rng, batch, page, wide, num_pages, fill)
    new = new(lens) if callable(new) else new
    free = had if free is None else min(free, had)
    n_rows = sum(max(n, 0) for n in new) if n_rows is None else n_rows
    p = Plan(page, lens, table, stack, free, n_rows)
    new_t = torch.tensor(new, dtype=torch.int32, device="cuda")
    p.call(new_t)
    p.check(S.plan_append(page, new, lens, table, stack, free, n_rows))
    return p


@pytest.mark.parametrize("batch", [1, 2, 33, 512, 513, 1100])
def test_decode_step(batch):
    rng = random.Random(batch)
    run_case(rng, batch, 128, 5, batch * 5, [1] * batch, None)


@pytest.mark.parametrize("seed", range(12))
def test_mixed_steps(seed):
    rng = random.Random(seed)
    batch, page, wide = rng.randint(1, 60), rng.choice([8, 16, 128]), rng.randint(2, 40)

    def new(lens):
        return [rng.choice([0, 1, -t, -rng.randint(0, t), rng.randint(0, wide * page - t)]) for t in lens]

    p = run_case(rng, batch, page, wide, batch * wide, new, None, free=rng.choice([None, 5, 40]))
    assert p.slots.numel() >= 0


def test_large_prefill_over_many_blocks():
    rng = random.Random(5)
    batch, wide = 17, 300
    run_case(rng, batch, 128, wide, batch * wide, [rng.randint(0, 20000) for _ in range(batch)], 200009, fill=0.2)


def test_one_long_sequence():
    run_case(random.Random(6), 1, 8, 40000, 40000, [300001], None, fill=0.01)


def test_too_few_pages_refuses_whole_sequences():
    rng = random.Random(7)
    p = run_case(rng, 9, 8, 20, 200, [20] * 9, None, free=10)
    taken = p.taken.cpu().numpy()
    assert 0 < (taken > 0).sum() < 9


def test_rows_behind_the_last_sequence_and_zero_rows():
    rng = random.Random(8)
    run_case(rng, 3, 128, 4, 12, [5, 0, 7], 40)
    run_case(rng, 3, 128, 4, 12, [0, 0, 0], 0)
    run_case(rng, 4, 8, 6, 24, lambda lens: [-t for t in lens], 0)


@pytest.mark.parametrize("new,lens", [([200, 1], [10, 10]), ([-11, 3], [10, 10]), ([1, 1], [-4, 10]), ([1, 1], [33, 3])])
def test_lengths_out_of_range_are_refused_and_reported(new, lens):
    table = [[0, 1, -1, -1], [2, 3, -1, -1]]
    stack = [4, 5, 6, 7, -1, -1, -1, -1]
    p = Plan(8, lens, table, stack, 4, 210)
    p.call(torch.tensor(new, dtype=torch.int32, device="cuda"))
    ref = S.plan_append(8, new, lens, table, stack, 4, 210)
    assert ref["fault"]
    p.check(ref)


def test_rows_past_the_end_are_refused_and_reported():
    rng = random.Random(9)
    p = run_case(rng, 4, 8, 20, 80, [5, 9, 5, 2], 15)
    assert p.taken.tolist() == [5, 9, 0, 0]


def test_a_bad_stack_is_reported_and_touches_nothing_outside():
    # a count above the pool is taken as 0, a page number outside the pool gives slot -1
    p = Plan(8, [0], [[-1, -1]], [1, 0], 3, 4)
    p.call(torch.tensor([4], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert P.palu_get_device_status(p.ws)[0] == 7 and p.slots.tolist() == [-1] * 4 and int(p.free) == 0
    p = Plan(8, [0], [[-1, -1]], [1, 9], 2, 4)
    p.call(torch.tensor([4], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert P.palu_get_device_status(p.ws)[0] == 7 and p.slots.tolist() == [-1] * 4


def test_dropping_restores_the_stack_and_outputs_are_optional():
    rng = random.Random(10)
    lens, table, stack, free = make_state(rng, 40, 8, 12, 700)
    p = Plan(8, lens, table, stack, free, 40 * 30)
    new = torch.tensor([rng.randint(0, 30) for _ in range(40)], dtype=torch.int32, device="cuda")
    p.call(new, starts=False)
    p.call(-new, starts=False)
    torch.cuda.synchronize()
    assert (p.lens.tolist(), p.table.tolist(), p.stack.tolist(), int(p.free)) == (lens, table, stack, free)


def test_captured_steps_replay():
    """Twenty decode steps from one captured graph equal twenty steps of the oracle."""
    rng = random.Random(11)
    lens, table, stack, free = make_state(rng, 30, 8, 12, 400)
    p = Plan(8, lens, table, stack, free, 30)
    new = torch.ones(30, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        p.call(new)
    for _ in range(20):
        graph.replay()
        r = S.plan_append(8, [1] * 30, lens, table, stack, free, 30)
        p.check(r)
        lens, table, stack, free = r["seq_lens"], r["page_table"], r["free_pages"], r["num_free"]


def test_another_stream():
    rng = random.Random(12)
    lens, table, stack, free = make_state(rng, 30, 8, 12, 400)
    p = Plan(8, lens, table, stack, free, 30)
    new = torch.ones(30, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.call(new, stream=s)
    p.check(S.plan_append(8, [1] * 30, lens, table, stack, free, 30))


def test_many_short_sequences():
    """Rows of one thread belong to several sequences, empty ones between them."""
    rng = random.Random(11)
    batch, wide = 8192, 4
    new = [rng.choice([0, 0, 0, 1, 1, 2, 3, 40]) for _ in range(batch // 2)] + [rng.choice([0, 30]) for _ in range(batch // 2)]
    assert sum(new) > 148 * 512
    run_case(rng, batch, 16, wide, batch * wide, new, None, fill=0.3)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_outputs_that_start_anywhere(offset):
    rng = random.Random(12)
    lens, table, stack, had = make_state(rng, 5, 24, 2000, 10000, 0.2)
    new = [19999, 0, 30001, 17, 40000]
    n = sum(new) + 6
    p = Plan(24, lens, table, stack, had, n)
    p.slots, p.positions = (torch.full((n + 4,), 77, dtype=torch.int32, device="cuda")[offset:offset + n] for _ in range(2))
    p.call(torch.tensor(new, dtype=torch.int32, device="cuda"))
    p.check(S.plan_append(24, new, lens, table, stack, had, n))


@pytest.mark.parametrize("page,wide", [(1000000, 2147), (524296, 4096), (524296, 4095), (8, 3000), (40, 3000), (1 << 20, 2047)])
def test_quotients_by_any_page_size(page, wide):
    """Positions up to the last below 2^31 that the page size allows."""
    cap = page * wide
    if cap >= 2 ** 31:                                # 524296·4096 = 2^31 + 32768: past the documented limit
        p = Plan(page, [0], [[-1] * wide], list(range(wide)), wide, 1)
        with pytest.raises(P.PaluError):
            p.call(torch.ones(1, dtype=torch.int32, device="cuda"))
        return
    for length, new in ((cap - 90001, 90001), (cap - 7 * page // 3, 300), (page - 1, 2), (0, 1)):
        had = -(-length // page)
        table = [list(range(had)) + [-1] * (wide - had)]
        stack = list(range(wide - 1, had - 1, -1)) + [-1] * had
        n = min(new, cap - length)
        if length < 0:
            continue
        p = Plan(page, [length], table, stack, wide - had, n)
        p.call(torch.tensor([n], dtype=torch.int32, device="cuda"))
        p.check(S.plan_append(page, [n], [length], table, stack, wide - had, n))


@pytest.mark.parametrize("rows", [0, 90000])
def test_batches_around_the_default_shared_memory(rows):
    """In a process of its own: no larger call has raised the kernel's limit before."""
    code = f"""
import random, sys
sys.path[:0] = {[os.path.dirname(os.path.abspath(__file__)), os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]!r}
import test_gpu_plan_append as T
for batch in (3054, 3055, 3071, 3075, 3054):
    new = [1] * batch
    new[7] += {rows}
    T.run_case(random.Random(batch), batch, 8, 4 if not {rows} else 12000, 20000 if {rows} else batch * 4, new, None, fill=0.3 if not {rows} else 1e-4)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("pages", [3, 700])
def test_bad_pages_given_back_stay_off_the_stack(pages):
    rng = random.Random(13)
    table = [rng.sample(range(3 * pages), pages), [], list(range(3 * pages, 4 * pages))]
    table[1] = [p for p in range(3 * pages) if p not in set(table[0])][:pages]
    used = set(sum(table, []))
    stack = [p for p in range(4 * pages) if p not in used]
    had = len(stack)
    stack += [-1] * (4 * pages - had)
    for b in range(3):
        for lp in rng.sample(range(pages), 1 + pages // 5):
            table[b][lp] = rng.choice([-1, -5, 4 * pages, 2 ** 31 - 1])
    lens, new = [8 * pages] * 3, [-8 * pages, 0, -8 * (pages - 1)]
    p = Plan(8, lens, table, stack, had, 0)
    p.call(torch.tensor(new, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    ref = S.plan_append(8, new, lens, table, stack, had, 0)
    assert ref["fault"] and P.palu_get_device_status(p.ws)[0] == 7
    assert int(p.free) == ref["num_free"] and p.stack.tolist()[:ref["num_free"]] == ref["free_pages"][:ref["num_free"]]
    assert p.table.tolist() == ref["page_table"] and p.lens.tolist() == ref["seq_lens"]
