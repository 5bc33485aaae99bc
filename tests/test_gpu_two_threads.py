"""Calls from host threads of their own: a thread that has made no CUDA call before, and two that call one
entry point with different sizes, each on a stream and a workspace of its own."""
import threading

import pytest
import torch

from rank_kv_cache_palu_b200 import api as P

pytestmark = pytest.mark.gpu


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


def plan(large):
    batch = 8192 if large else 4096
    args = (i32(batch), i32(batch), i32(batch, 1), i32(8), i32(1), i32(0), i32(0), None, None,
            torch.zeros(P.palu_plan_workspace_size(batch), dtype=torch.uint8, device="cuda"))
    return lambda st: P.palu_plan_append(8, *args, stream=st)


def select(large):
    cfg = P.make_config(4, 64, 4, 64, 64, 8, 10000.0, "bf16")
    wide = 32768 if large else 16384
    ws = torch.zeros(P.palu_select_workspace_size(cfg, 1, 1, wide), dtype=torch.uint8, device="cuda")
    args = (torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda"), i32(1, 1),
            torch.zeros(512, dtype=torch.bfloat16, device="cuda"), None, i32(1, wide), i32(1, fill=5), 1, 0, 0,
            i32(1, 1, 1, 1), i32(1, 1, 1), None, ws)
    return lambda st: P.palu_select_pages(cfg, *args, stream=st)


def layer(large, rope, ranks, act="bf16"):
    rank = ranks[large]
    cfg = P.make_config(4, 128, 4, rank, 128, 128, rope, act)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[act]
    zero = lambda n: torch.zeros(n, dtype=dt, device="cuda")
    return cfg, zero(128 * rank), zero(128 * 128), zero(rank * 512), zero(128 * 512), zero


def bounds(large):
    cfg, zk, _, Bk, _, zero = layer(large, 10000.0, (64, 256))
    ws = torch.zeros(P.palu_page_bounds_workspace_size(cfg, 1, 1), dtype=torch.uint8, device="cuda")
    args = (None, zk, None, None, i32(1, 1), i32(1, fill=5), 1, Bk, zero(1024), ws)
    return lambda st: P.palu_page_bounds(cfg, *args, stream=st)


def attend(large, rope=10000.0, ranks=(64, 256)):
    cfg, zk, zv, Bk, Bv, zero = layer(large, rope, ranks)
    ws = torch.zeros(P.palu_decode_pages_workspace_size(cfg, 1, 1, 1), dtype=torch.uint8, device="cuda")
    args = (zero(512).view(1, 1, 4, 128), i32(1, 1), zk, zv, None, None, None, i32(1, 1), i32(1, fill=5),
            i32(1, 1, 1, 1), i32(1, 1, 1, fill=1), 1, Bk, Bv, zero(512).view(1, 1, 4, 128), None, ws)
    return lambda st: P.palu_decode_attn_pages(cfg, *args, stream=st)


def attend_norope(large):
    return attend(large, 0.0, (64, 512))


def dense(large, rope=10000.0, ranks=(64, 256), act="bf16"):
    cfg, zk, zv, Bk, Bv, zero = layer(large, rope, ranks, act)
    ws = torch.zeros(P.palu_decode_workspace_size(cfg, 1, 1), dtype=torch.uint8, device="cuda")
    args = (zero(512).view(1, 4, 128), i32(1), zk, zv, None, None, None, i32(1, 1), i32(1, fill=5), 1, Bk, Bv,
            zero(512).view(1, 4, 128), None, ws)
    return lambda st: P.palu_decode_attn(cfg, *args, stream=st)


def dense_norope(large):
    return dense(large, 0.0, (64, 512))


def dense_f32(large):
    return dense(large, 10000.0, (448, 512), "f32")


def compress(large):
    cfg, n, d = P.make_config(4, 128, 4, 256, 128, 128, 10000.0, "bf16"), 128 if large else 16, 256
    zero = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(P.palu_compress_workspace_size(cfg, n, d), dtype=torch.uint8, device="cuda")
    args = (zero(n, d), zero(d, 256), zero(d, 128), i32(n, fill=-1), i32(n), zero(128 * 256), zero(128 * 128), None, None,
            None, 1, ws)
    return lambda st: P.palu_compress_append(cfg, *args, stream=st)


EVERY = [plan, select, bounds, attend, attend_norope, dense, dense_norope, dense_f32, compress]


@pytest.mark.parametrize("make", EVERY, ids=lambda f: f.__name__)
def test_a_thread_of_no_cuda_call_before(make):
    call, stream, failed = make(True), torch.cuda.Stream(), []
    torch.cuda.synchronize()

    def work():
        try:
            call(stream)
        except P.PaluError as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]


def raw(make, large, stream, monkeypatch):
    """The library call that make's call comes to, with its arguments: nothing of Python's between two."""
    call, lib, seen = make(large), P.load(), []

    class Recorder:
        def __getattr__(self, name):
            fn = getattr(lib, name)
            return lambda *a: seen.append((fn, a)) or fn(*a)

    with monkeypatch.context() as m:
        m.setattr(P, "load", Recorder)
        call(stream)
    return seen[-1] + (call,)


@pytest.mark.parametrize("make", EVERY, ids=lambda f: f.__name__)
def test_sizes_of_two_threads(make, monkeypatch):
    """None of two calls may lower what the other's launch is allowed."""
    calls, failed = [], []
    for large in (False, True):
        stream = torch.cuda.Stream()
        calls.append((stream, *raw(make, large, stream, monkeypatch)))
    torch.cuda.synchronize()

    def work(stream, fn, args, _):
        for n in range(5000):
            if fn(*args) != 0:
                failed.append(P.load().palu_last_cuda_error().decode())
                return
            if n % 256 == 255:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]
