"""The serving operators run together, as a drafting server uses them: plan the rows of a step,
append the latents, rebuild the bounds of the touched pages, pick pages, attend over them, verify the
drafts and drop the refused ones.  Each stage's outputs feed the next on the GPU; eager and captured."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from oracle import palu_oracle as O
from oracle import serving_oracle as S
from rank_kv_cache_palu_b200 import api as P
from rank_kv_cache_palu_b200.synth import TORCH_DTYPE, WORKLOADS, normal_tensor

pytestmark = pytest.mark.gpu
PAGE, MODEL = 128, 256
KINDS = {
    "rope_bf16": dataclasses.replace(WORKLOADS["7b_bf16_r256v128_b1_t4k"], num_heads=8),
    "norope_f16": dataclasses.replace(WORKLOADS["7b_bf16_r256v128_b1_t4k"], num_heads=8, rope_base=0.0, act_dtype="f16",
                                      latent_dtype="f16"),
    "int4": dataclasses.replace(WORKLOADS["7b_int4_r256_b8_t32k"], num_heads=8),
    "tiny_f32": dataclasses.replace(WORKLOADS["tiny_f32"]),
}


class Server:
    """One layer of a server: cache, page state, bounds and the workspaces it keeps."""

    def __init__(self, w, batch=3, wide=8, drafts=3, keep=4, vocab=500):
        self.w, self.batch, self.wide, self.Q, self.keep, self.vocab = w, batch, wide, drafts, keep, vocab
        self.act = TORCH_DTYPE[w.act_dtype]
        self.cfg = c = P.make_config(w.num_heads, w.head_dim, w.group_size, w.rank_k, w.rank_v, PAGE, w.rope_base,
                                     w.act_dtype, w.latent_dtype)
        G, W = w.groups, w.width
        self.pages = batch * wide + 2
        self.cache = P.LatentCache.allocate(c, self.pages, fill=0xFF)          # NaN wherever nothing was written
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")
        self.table, self.lens = z(batch, wide) - 1, z(batch)
        self.stack = torch.randperm(self.pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.free = z(1) + self.pages
        self.bounds = z(self.pages, G, 2, W, t=self.act)
        rand = lambda tag, *s, std=1.0: normal_tensor(7, tag, s, w.act_dtype, std).cuda()
        self.A_k, self.A_v = rand("A_k", MODEL, G * w.rank_k, std=MODEL ** -.5), rand("A_v", MODEL, G * w.rank_v, std=MODEL ** -.5)
        self.B_k, self.B_v = rand("B_k", G, w.rank_k, W, std=w.rank_k ** -.5), rand("B_v", G, w.rank_v, W, std=w.rank_v ** -.5)
        self.head = torch.randn((w.num_heads * w.head_dim, vocab), generator=torch.Generator().manual_seed(2)).cuda()
        ws = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
        rows = 6 * PAGE * batch
        self.ws_plan, self.ws_verify = ws(P.palu_plan_workspace_size(batch)), ws(P.palu_verify_workspace_size(batch, drafts, vocab))
        self.ws_append = ws(max(P.palu_compress_workspace_size(c, n, MODEL) for n in (batch * drafts, 887, rows)))
        self.ws_bounds = ws(P.palu_page_bounds_workspace_size(c, batch, wide))
        self.ws_select = ws(P.palu_select_workspace_size(c, batch, drafts, wide))
        self.ws_attend = ws(P.palu_decode_pages_workspace_size(c, batch, drafts, keep))
        self.step_table = z(batch, wide)
        self.before, self.row_starts, self.taken = z(batch), z(batch + 1), z(batch)
        self.lists, self.counts = z(batch, drafts, G, keep), z(batch, drafts, G)
        self.out = z(batch, drafts, w.num_heads, w.head_dim, t=self.act)
        self.lse = z(batch, drafts, w.num_heads, t=torch.float32)
        self.tokens, self.accepted, self.rollback = z(batch, drafts + 1), z(batch), z(batch)
        self.rows = {n: (z(n), z(n)) for n in (batch * drafts, rows)}

    def append(self, new, x):
        """Plan, compress and bound the rows of x."""
        slots, positions = self.rows[x.shape[0]] if x.shape[0] in self.rows else \
            tuple(torch.zeros(x.shape[0], dtype=torch.int32, device="cuda") for _ in range(2))
        self.before.copy_(self.lens)
        P.palu_plan_append(PAGE, new, self.lens, self.table, self.stack, self.free, slots, positions, self.row_starts,
                           self.taken, self.ws_plan)
        P.palu_compress_append(self.cfg, x, self.A_k, self.A_v, slots, positions, self.cache.zk, self.cache.zv,
                               self.cache.zks, self.cache.zvs, None, self.pages, self.ws_append)
        self.bound(self.before)
        return slots, positions

    def bound(self, first):
        P.palu_page_bounds(self.cfg, first, self.cache.zk, self.cache.zks, None, self.table, self.lens, self.pages,
                           self.B_k, self.bounds, self.ws_bounds)

    def step(self, new, x, q, drafts, draft_probs, u_accept, u_sample):
        """One drafting step: q [batch][Q][H][d] of the Q appended tokens."""
        _, positions = self.append(new, x)
        q_pos = positions.view(self.batch, self.Q)
        P.palu_select_pages(self.cfg, q, q_pos, self.bounds, None, self.table, self.lens, self.pages, 1, 1, self.lists,
                            self.counts, None, self.ws_select)
        P.palu_decode_attn_pages(self.cfg, q, q_pos, self.cache.zk, self.cache.zv, self.cache.zks, self.cache.zvs, None,
                                 self.table, self.lens, self.lists, self.counts, self.pages, self.B_k, self.B_v, self.out,
                                 self.lse, self.ws_attend)
        self.step_table.copy_(self.table)          # as the step saw it, before refused drafts give pages back
        # a stand-in for the rest of the model; the step's first token is the last accepted one
        logits = self.out.float().flatten(2) @ self.head
        self.probs = torch.softmax(logits, -1)
        P.palu_verify_drafts(self.probs, draft_probs, drafts, None, u_accept, u_sample, self.tokens[:, :self.Q],
                             self.accepted, self.rollback, self.ws_verify)
        P.palu_plan_append(PAGE, self.rollback, self.lens, self.table, self.stack, self.free, *self.rows_none(), None, None,
                           self.ws_plan)
        self.bound(self.lens)

    def rows_none(self):
        if not hasattr(self, "none"):
            self.none = tuple(torch.zeros(0, dtype=torch.int32, device="cuda") for _ in range(2))
        return self.none

    def good(self):
        torch.cuda.synchronize()
        for ws in (self.ws_plan, self.ws_append, self.ws_bounds, self.ws_select, self.ws_attend, self.ws_verify):
            assert P.palu_get_device_status(ws) == (0, 0)


def make(kind, drafts=3, keep=4):
    s = Server(KINDS[kind], drafts=drafts, keep=keep)
    s.tokens = torch.zeros((s.batch, drafts), dtype=torch.int32, device="cuda")
    s.ws_verify = torch.zeros(P.palu_verify_workspace_size(s.batch, drafts - 1, s.vocab), dtype=torch.uint8, device="cuda")
    prompt = [500, 127, 260]
    x = normal_tensor(3, "prompt", (sum(prompt), MODEL), s.w.act_dtype).cuda()
    s.append(torch.tensor(prompt, dtype=torch.int32, device="cuda"), x)
    return s, prompt, x


def inputs(s, i):
    w, D = s.w, s.Q - 1
    g = torch.Generator().manual_seed(100 + i)
    x = normal_tensor(50 + i, "x", (s.batch * s.Q, MODEL), w.act_dtype).cuda()
    q = normal_tensor(50 + i, "q", (s.batch, s.Q, w.num_heads, w.head_dim), w.act_dtype).cuda()
    draft = torch.softmax(torch.randn((s.batch, D, s.vocab), generator=g) * 2, -1)
    tokens = torch.multinomial(draft.view(-1, s.vocab), 1, generator=g).view(s.batch, D).to(torch.int32)
    return dict(x=x, q=q, drafts=tokens.cuda(), draft_probs=draft.cuda(), u_accept=(torch.rand((s.batch, D), generator=g) * 0.3).cuda(),
                u_sample=torch.rand(s.batch, generator=g).cuda())


def state(s):
    torch.cuda.synchronize()
    # stale stack entries above the top and the bounds of free pages are nobody's
    live = sorted(int(p) for p in s.table.flatten().tolist() if p >= 0)
    return [s.lens.clone(), s.table.clone(), s.free.clone(), s.stack[:int(s.free)].clone(), s.bounds[live].clone(),
            s.out.clone(), s.lse.clone(), s.tokens.clone(), s.accepted.clone(), s.lists.clone()]


@pytest.mark.parametrize("kind", list(KINDS))
def test_steps_against_the_oracle(kind):
    s, prompt, x0 = make(kind)
    w = s.w
    G = w.groups
    f64 = lambda t: t.double().cpu().numpy()
    Ak, Av, Bk, Bv = f64(s.A_k), f64(s.A_v), f64(s.B_k), f64(s.B_v)
    rows = np.split(f64(x0), np.cumsum(prompt)[:-1])
    new = torch.full((s.batch,), s.Q, dtype=torch.int32, device="cuda")

    def latents(x, A, r):
        if w.latent_dtype == "int4":
            z = (x @ A).astype(np.float32).reshape(len(x), G, r).transpose(1, 0, 2)
            return O.dequantize_int4(*O.quantize_int4(z), w.act_dtype)
        return O.compress(x, A, w.act_dtype).reshape(len(x), G, r).transpose(1, 0, 2)

    # rounding of the latents themselves (float32 sums round to another 16-bit or 4-bit neighbour now and
    # then) comes on top of the operator's own bounds: the step is held to the parity bar of the path
    tol = 1e-4 if w.act_dtype == "f32" else 1e-2 if w.latent_dtype != "int4" else 5e-2
    for i in range(3):
        d = inputs(s, i)
        lens = s.lens.tolist()
        s.step(new, **d)
        s.good()
        xs = f64(d["x"]).reshape(s.batch, s.Q, MODEL)
        for b in range(s.batch):
            all_x = np.concatenate([rows[b], xs[b]])
            assert len(rows[b]) == lens[b]
            T = lens[b] + s.Q
            zk, zv = latents(all_x, Ak, w.rank_k), latents(all_x, Av, w.rank_v)
            for j in range(s.Q):
                at = lens[b] + j
                n = -(-(at + 1) // PAGE)
                mine = [[p for p in l if p >= 0] for l in s.lists[b, j].tolist()]
                assert all(len(l) == min(s.keep, n) and l == sorted(set(l)) and l[0] == 0 and l[-1] == n - 1 for l in mine)
                ref, lse, _ = S.decode_attention_pages(f64(d["q"])[b, j], at, zk, zv, np.arange(T), Bk, Bv, w.group_size,
                                                       w.rope_base, mine, PAGE, True)
                got = f64(s.out)[b, j]
                assert np.max(np.abs(got - ref)) <= tol * np.max(np.abs(ref)), f"step {i} seq {b} query {j}"
            t, a = S.verify_drafts(f64(s.probs)[b], f64(d["draft_probs"])[b], d["drafts"][b].cpu().numpy(), s.Q - 1,
                                   d["u_accept"][b].cpu().numpy(), float(d["u_sample"][b]))
            assert (s.tokens[b].tolist(), int(s.accepted[b])) == (t, a)
            rows[b] = all_x[:lens[b] + 1 + a]          # the refused drafts are dropped
            assert int(s.lens[b]) == len(rows[b])
        # the kept pages' bounds are those of a pool built anew
        kept = s.bounds.clone()
        s.bounds.fill_(3.0)
        s.bound(None)
        torch.cuda.synchronize()
        live = [p for p in s.table.flatten().tolist() if p >= 0]
        assert torch.equal(kept[live].view(torch.uint8), s.bounds[live].view(torch.uint8))
        assert sorted(live + s.stack[:int(s.free)].tolist()) == list(range(s.pages))


@pytest.mark.parametrize("kind", ["rope_bf16", "norope_f16", "int4"])
def test_every_page_kept_equals_the_dense_step(kind):
    """With room for every page the step is palu_decode_attn_multi's, up to its 16-bit softmax weights:
    2^-8 (bf16) or 2^-11 (f16) of Σ p|v| <= 3 max|out| here, and a final rounding on each side."""
    s, _, _ = make(kind, keep=8)
    d = inputs(s, 0)
    s.step(torch.full((s.batch,), s.Q, dtype=torch.int32, device="cuda"), **d)
    s.good()
    w = s.w
    # the step has dropped its refused drafts; the pages still hold their latents
    lens = s.before + s.Q
    q_pos = s.before[:, None] + torch.arange(s.Q, device="cuda", dtype=torch.int32)
    out, lse = torch.empty_like(s.out), torch.empty_like(s.lse)
    ws = torch.zeros(P.palu_decode_multi_workspace_size(s.cfg, s.batch, s.Q, s.wide), dtype=torch.uint8, device="cuda")
    P.palu_decode_attn_multi(s.cfg, d["q"], q_pos.contiguous(), s.cache.zk, s.cache.zv, s.cache.zks, s.cache.zvs, None,
                             s.step_table, lens, s.pages, s.B_k, s.B_v, out, lse, ws)
    torch.cuda.synchronize()
    half = 2.0 ** -8 if w.act_dtype == "bf16" else 2.0 ** -11
    assert float((out.double() - s.out.double()).abs().max()) <= 5 * half * float(out.abs().max())
    assert float((lse - s.lse).abs().max()) <= 2 * half


@pytest.mark.parametrize("kind", ["rope_bf16", "norope_f16", "int4", "tiny_f32"])
def test_captured_steps_equal_eager_ones(kind):
    eager, captured = make(kind)[0], make(kind)[0]
    new = torch.full((eager.batch,), eager.Q, dtype=torch.int32, device="cuda")
    held = inputs(captured, 0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    # cuBLAS wants a first call outside the capture
    _ = captured.out.float().flatten(2) @ captured.head
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured.step(new, **held)
    for i in range(4):
        d = inputs(eager, i)
        eager.step(new, **d)
        for k in held:
            held[k].copy_(d[k])
        graph.replay()
        eager.good()
        captured.good()
        for x, y in zip(state(eager), state(captured)):
            assert torch.equal(x.view(torch.uint8) if x.dtype.is_floating_point else x,
                               y.view(torch.uint8) if y.dtype.is_floating_point else y)


def test_two_graphs_with_workspaces_of_their_own_run_at_once():
    servers = [make("rope_bf16")[0] for _ in range(2)]
    alone = make("rope_bf16")[0]
    new = torch.full((alone.batch,), alone.Q, dtype=torch.int32, device="cuda")
    d = inputs(alone, 0)
    alone.step(new, **d)
    want = state(alone)
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in servers:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step(new, **d)
        graphs.append(g)
    torch.cuda.synchronize()
    for g, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for s in servers:
        s.good()
        for x, y in zip(want, state(s)):
            assert torch.equal(x.view(torch.uint8) if x.dtype.is_floating_point else x,
                               y.view(torch.uint8) if y.dtype.is_floating_point else y)
