"""palu_verify_drafts on the GPU against the CPU oracle: tokens and counts are whole numbers and equal."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from rank_kv_cache_palu_b200 import api as P

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(batch, D, V, dtype, seed=0, pad=0, near=0.5, drafter=True, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((batch, D + 1, V), generator=g) * sharp
    close = logits[:, :D] + near * torch.randn((batch, D, V), generator=g)
    target = torch.zeros((batch, D + 1, V + pad), dtype=DT[dtype])
    target[..., :V] = torch.softmax(logits, -1).to(DT[dtype])
    draft = torch.full((batch, D, V + pad), 5.0, dtype=DT[dtype])
    draft[..., :V] = torch.softmax(close, -1).to(DT[dtype])
    noise = torch.empty((batch, D, V)).exponential_(generator=g)
    tokens = (torch.softmax(close, -1) / noise).argmax(-1).to(torch.int32) if D else \
        torch.zeros((batch, 0), dtype=torch.int32)
    lens = torch.randint(0, D + 1, (batch,), generator=g, dtype=torch.int32)
    u_accept, u_sample = torch.rand((batch, D), generator=g), torch.rand((batch,), generator=g)
    return dict(target=target, draft=draft if drafter else None, tokens=tokens, lens=lens, ua=u_accept, us=u_sample,
                V=V)


def run(c, lens=True, status=0, ws=None, twice=True):
    batch, n = c["target"].shape[:2]
    dev = lambda t: None if t is None else t.cuda()
    out = torch.full((batch, n), 99, dtype=torch.int32, device="cuda")
    acc, back = (torch.full((batch,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    if ws is None:
        ws = torch.zeros(P.palu_verify_workspace_size(batch, n - 1, c["V"]), dtype=torch.uint8, device="cuda")
    target, draft = dev(c["target"])[..., :c["V"]], dev(c["draft"])
    args = (target, None if draft is None else draft[..., :c["V"]], dev(c["tokens"]), dev(c["lens"]) if lens else None,
            dev(c["ua"]), dev(c["us"]), out, acc, back, ws)
    P.palu_verify_drafts(*args)
    first = out.clone(), acc.clone(), back.clone()
    if twice:
        P.palu_verify_drafts(*args)
    torch.cuda.synchronize()
    assert P.palu_get_device_status(ws)[0] == status
    for x, y in zip(first, (out, acc, back)):
        assert torch.equal(x, y)
    return out.cpu().numpy(), acc.cpu().numpy(), back.cpu().numpy()


def check(c, lens=True, **kw):
    out, acc, back = run(c, lens, **kw)
    batch, n = c["target"].shape[:2]
    V = c["V"]
    for b in range(batch):
        want = int(c["lens"][b]) if lens else n - 1
        want = min(max(want, 0), n - 1)
        t = c["target"][b, :, :V].double().numpy()
        d = None if c["draft"] is None else c["draft"][b, :, :V].double().numpy()
        ref, a = S.verify_drafts(t, d, c["tokens"][b].numpy(), want, c["ua"][b].numpy(), float(c["us"][b]))
        assert (out[b].tolist(), int(acc[b]), int(back[b])) == (ref, a, a - want), f"sequence {b}"
    return acc


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("batch,D,V", [(1, 1, 1), (3, 2, 7), (5, 4, 1000), (7, 7, 2049), (2, 3, 32000), (40, 5, 5003)])
def test_sizes(dtype, batch, D, V):
    check(make(batch, D, V, dtype, seed=V + D))


@pytest.mark.parametrize("dtype,pad", [("bf16", 1), ("f16", 3), ("f32", 1), ("bf16", 8)])
def test_padded_rows(dtype, pad):
    check(make(6, 3, 4099, dtype, seed=pad, pad=pad))


def test_certain_drafts_and_no_lengths():
    c = make(12, 4, 3001, "f32", seed=3, drafter=False, sharp=6.0)
    c["tokens"] = c["target"][:, :4, :3001].argmax(-1).to(torch.int32)
    acc = check(c, lens=False)
    assert acc.max() > 0
    check(c)


def test_no_drafts_samples_the_target():
    c = make(9, 0, 2500, "f32", seed=4)
    check(c, lens=False)


def test_most_drafts_and_all_accepted():
    c = make(3, 32, 300, "f32", seed=5, near=0.0)
    c["ua"][:] *= 0.999
    acc = check(c, lens=False)
    assert (acc == 32).all()


@pytest.mark.parametrize("u", [0.0, 1 - 2.0 ** -24])
def test_ends_of_the_running_sum(u):
    c = make(5, 2, 4097, "f32", seed=6)
    c["us"][:] = u
    check(c)


def test_rows_without_weight_and_bad_entries():
    c = make(6, 1, 5000, "f32", seed=7)
    t, d = c["target"], c["draft"]
    t[0] = 0.0                                   # nothing to draw: token -1
    t[1, :, 10] = float("nan")
    d[1, :, 11] = float("nan")
    t[2, :, 20] = float("inf")
    t[3, :, 30] = -1.0
    d[4] = 1.0                                   # p <= q everywhere: the draw falls back to p
    c["lens"][:] = 1
    c["ua"][:] = 0.9999
    out, acc, back = run(c)
    assert out[0].tolist() == [-1, -1] and out[0][1] == -1
    check(c)


def test_one_positive_entry_in_each_chunk_border():
    for v in (0, 2047, 2048, 4095, 4096, 8190):
        c = make(1, 0, 8191, "f32", seed=8)
        c["target"][:] = 0
        c["target"][0, 0, v] = 0.25
        c["us"][:] = 0.5
        assert check(c, lens=False) == 0
        assert run(c, lens=False)[0][0, 0] == v


def test_bad_tokens_and_lengths_are_reported():
    c = make(3, 2, 500, "f32", seed=9)
    c["tokens"][0, 0], c["tokens"][1, 1] = 500, -1
    c["lens"][:] = 2
    c["ua"][:] = 0.0
    check(c, status=7)
    c = make(3, 2, 500, "f32", seed=10)
    c["lens"] = torch.tensor([5, -3, 1], dtype=torch.int32)
    check(c, status=7)


def test_one_workspace_serves_calls_of_any_size_it_holds():
    ws = torch.zeros(P.palu_verify_workspace_size(50, 3, 9000), dtype=torch.uint8, device="cuda")
    for batch, V in ((50, 9000), (2, 9000), (50, 300), (1, 8000), (50, 9000)):
        check(make(batch, 3, V, "bf16", seed=batch), ws=ws)


def test_captured_call_follows_its_inputs():
    c = make(4, 3, 9001, "f32", seed=11)
    dev = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    out = torch.zeros((4, 4), dtype=torch.int32, device="cuda")
    acc = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(P.palu_verify_workspace_size(4, 3, 9001), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.palu_verify_drafts(dev["target"], dev["draft"], dev["tokens"], dev["lens"], dev["ua"], dev["us"], out, acc,
                             None, ws)
    for seed in (12, 13):
        d = make(4, 3, 9001, "f32", seed=seed)
        for k in dev:
            dev[k].copy_(d[k])
        graph.replay()
        torch.cuda.synchronize()
        for b in range(4):
            ref, a = S.verify_drafts(d["target"][b].double().numpy(), d["draft"][b].double().numpy(),
                                     d["tokens"][b].numpy(), int(d["lens"][b]), d["ua"][b].numpy(), float(d["us"][b]))
            assert (out[b].tolist(), int(acc[b])) == (ref, a)


@pytest.mark.parametrize("dtype,batch,V", [("bf16", 2, 1000003), ("f32", 1, 2 ** 21)])
def test_large_vocabularies(dtype, batch, V):
    """More groups than the drawing CTA keeps sums of."""
    c = make(batch, 2, V, dtype, seed=20)
    for u in (0.001, 0.7, 0.99999):
        c["us"][:] = u
        check(c, twice=False)


def test_the_largest_batch():
    check(make(8192, 1, 300, "f32", seed=21), twice=False)
