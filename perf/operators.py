"""Cases of the operators around the latent cache: planning a step's pages and slots, checking
drafted tokens, and attention over the pages that a cheap bound selects.

Five operators, each reached through ``rank_kv_cache_palu_b200.api`` where ``own`` is true and
written in elementary torch operations where it is false:

  plan     palu_plan_append        pages, slots and positions of the tokens a step appends
  verify   palu_verify_drafts      drafted tokens against the target's probabilities
  bounds   palu_page_bounds        per page and channel, the range of the rebuilt, rotated keys
  select   palu_select_pages       the pages of largest score bound, for each query and head group
  attend   palu_decode_attn_pages  a decode step over the selected pages only

Formulas (P tokens per page, head group g with latents z_k, z_v and factors B_k, B_v):
  keys      k_t = R(pos_t) (z_k,t B_k)              R: rotate-half RoPE, the identity at base 0
  bounds    lo = min_t k_t, hi = max_t k_t over the page's cached tokens, rounded outwards
  score     max over the group's heads h of Σ_c max(q'_h,c lo_c, q'_h,c hi_c), q' = R(q_pos) q
  attend    softmax over the listed pages' tokens of q'·k_t / √d_h, values (p·z_v) B_v
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# (heads, head_dim, heads per group, key rank, value rank)
SHAPES = {
    "7b": (32, 128, 4, 256, 128),        # the 7B-shaped layer of the benchmark
    "7b_r256": (32, 128, 4, 256, 256),   # the same with value rank 256 (int4 latents need it)
    "half": (16, 128, 2, 128, 128),      # half the heads, two per group
    "tiny": (8, 64, 4, 64, 64),          # the small float32 layer of the parity tests
}
PAGE = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a full server: every request appends one token, few cross a page border
        {"name": "plan_decode", "op": "plan", "batch": 256, "tokens": 256, "context": 4096, "kind": "decode",
         "spare": 0},
        # a prefill step: 64 ragged prompts, half a million tokens, some finished requests leave
        {"name": "plan_prefill", "op": "plan", "batch": 64, "tokens": 500009, "context": 2000, "kind": "mixed",
         "spare": 5},
        # one interactive request checking 3 drafted tokens
        {"name": "verify_one", "op": "verify", "batch": 1, "drafts": 3, "vocab": 32000, "dtype": "f32",
         "drafter": "probs", "pad": 0},
        # a batch checking up to 7 drafted tokens each over a large vocabulary whose rows are padded
        {"name": "verify_batch", "op": "verify", "batch": 64, "drafts": 7, "vocab": 128003, "dtype": "bf16",
         "drafter": "probs", "pad": 61},
        # a decode step: the page that got each request's new token
        {"name": "bounds_decode", "op": "bounds", "shape": "7b", "act": "bf16", "lat": "bf16", "rope": 10000.0,
         "batch": 16, "context": 16384, "span": 1, "explicit": False, "short": False},
        # the prefill of an 8192-token prompt
        {"name": "bounds_prefill", "op": "bounds", "shape": "7b", "act": "bf16", "lat": "bf16", "rope": 10000.0,
         "batch": 1, "context": 8192, "span": 64, "explicit": False, "short": False},
        # one long request
        {"name": "select_one", "op": "select", "shape": "7b", "act": "bf16", "rope": 10000.0, "batch": 1,
         "context": 65536, "queries": 1, "keep": 32, "short": False},
        # a batch of long requests, ragged, an empty and a one-token one among them
        {"name": "select_batch", "op": "select", "shape": "7b", "act": "bf16", "rope": 10000.0, "batch": 16,
         "context": 65536, "queries": 1, "keep": 64, "short": True},
        # one request of 16k tokens over 16 of its 128 pages
        {"name": "attend_one", "op": "attend", "shape": "7b", "act": "bf16", "lat": "bf16", "rope": 10000.0,
         "batch": 1, "context": 16384, "queries": 1, "keep": 16, "explicit": False, "short": False},
        # 16 requests of 64k tokens over a sixteenth of their pages
        {"name": "attend_batch", "op": "attend", "shape": "7b", "act": "bf16", "lat": "bf16", "rope": 10000.0,
         "batch": 16, "context": 65536, "queries": 1, "keep": 32, "explicit": False, "short": False},
        # the layer without rotary embedding, an eighth of the pages
        {"name": "attend_norope", "op": "attend", "shape": "7b", "act": "f16", "lat": "f16", "rope": 0.0,
         "batch": 16, "context": 65536, "queries": 1, "keep": 64, "explicit": False, "short": True},
        # four drafted tokens of each request, each with pages of its own, over 4-bit latents
        {"name": "attend_int4_drafts", "op": "attend", "shape": "7b_r256", "act": "f16", "lat": "int4",
         "rope": 10000.0, "batch": 8, "context": 32768, "queries": 4, "keep": 16, "explicit": False,
         "short": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _layer(rng):
    """A layer: shape, compute type, latent type and RoPE base that go together."""
    shape = rng.choice(["7b", "7b", "7b_r256", "half", "tiny"])
    act = "f32" if shape == "tiny" else rng.choice(["bf16", "f16"])
    lat = "int4" if shape == "7b_r256" and rng.random() < 0.5 else act
    return {"shape": shape, "act": act, "lat": lat, "rope": rng.choice([10000.0, 10000.0, 0.0])}


def draw(rng):
    op = rng.choice(["plan", "verify", "bounds", "select", "attend"])
    if op == "plan":
        kind = rng.choice(["decode", "mixed"])
        batch = _log(rng, 1, 512)
        tokens = batch if kind == "decode" else _log(rng, batch, 400000)
        return {"op": op, "batch": batch, "tokens": tokens, "context": _log(rng, 8, 8000), "kind": kind,
                "spare": rng.choice([0, 0, 7])}
    if op == "verify":
        return {"op": op, "batch": _log(rng, 1, 60), "drafts": rng.randint(1, 7), "vocab": _log(rng, 500, 120000),
                "dtype": rng.choice(["f32", "f16", "bf16"]), "drafter": rng.choice(["probs", "probs", "fixed"]),
                "pad": rng.choice([0, 0, 1, 8, 29])}
    layer = _layer(rng)
    small = layer["shape"] == "tiny"
    batch = _log(rng, 1, 8 if small else 16)
    short = batch >= 4 and rng.random() < 0.5
    if op == "bounds":
        span = 1 if rng.random() < 0.5 else _log(rng, 2, 8 if small else 64)
        batch = batch if span == 1 else min(batch, max(1, 64 // span))
        return {"op": op, **layer, "batch": batch, "context": _log(rng, span * PAGE, max(span * PAGE, 16384)) + 1,
                "span": span, "explicit": rng.random() < 0.25, "short": short and batch >= 4}
    queries = rng.choice([1, 1, 1, 2, 3, 4])
    if op == "select":
        layer.pop("lat")
        return {"op": op, **layer, "batch": batch, "context": _log(rng, 300, 60000), "queries": queries,
                "keep": _log(rng, 3, 64), "short": short}
    keep = _log(rng, 1, 4 if small else 32)
    return {"op": op, **layer, "batch": max(1, batch // queries), "context": _log(rng, 300, 4096 if small else 32768),
            "queries": queries, "keep": keep, "explicit": rng.random() < 0.2, "short": short and batch // queries >= 4}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _lens(case, rng, least):
    """Ragged lengths up to the context; with "short" an empty and a one-token sequence among them."""
    top = case["context"]
    lens = [rng.randint(max(1, least, int(0.8 * top)), max(1, least, top)) for _ in range(case["batch"])]
    if case["short"]:
        lens[0], lens[1] = 1, 0
    return lens


def _tables(lens, context, gen):
    """Page table over a shuffled pool that holds every sequence at its longest; unused entries are -1."""
    pages, wide = [-(-t // PAGE) for t in lens], -(-context // PAGE)
    total = len(lens) * wide + 2
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.full((len(lens), wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


def _pool(total, groups, rank, lat, gen):
    """Latents N(0, 1) in the cache's bytes, and int4 scales; the swizzle only moves iid entries about."""
    if lat != "int4":
        z = torch.randn((total * groups, PAGE * rank), generator=gen, device="cuda", dtype=TYPES[lat])
        return z.view(torch.uint8).view(-1), None
    n = total * groups * PAGE
    code = (torch.randn((n, rank), generator=gen, device="cuda", dtype=torch.float16) * 2.7).round_().clamp_(-7, 7)
    code = code.to(torch.int8).bitwise_and_(15).view(torch.uint8)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    wide = -(-2 * (rank // 32) // 16) * 8                   # fp16 scales per row, padded to 16 bytes
    scale = torch.rand((n, wide), generator=gen, device="cuda").mul_(0.2).add_(0.27).half()
    return packed.reshape(-1), scale.view(torch.uint8).reshape(-1)


def _factor(groups, rank, width, act, gen):
    return (torch.randn((groups, rank, width), generator=gen, device="cuda") / math.sqrt(rank)).to(TYPES[act])


def _positions(lens, table, total, explicit):
    """Positions 3t + 1 of token t in a position pool, or none: a token's position is then its index."""
    if not explicit:
        return None
    pool = torch.zeros((total + 1, PAGE), dtype=torch.int32, device="cuda")
    wide = table.shape[1]
    pos = (torch.arange(wide * PAGE, device="cuda", dtype=torch.int32) * 3 + 1).view(1, wide, PAGE)
    pool[torch.where(table >= 0, table, total).long()] = pos.expand(len(lens), wide, PAGE).contiguous()
    return pool[:total].contiguous()


def prepare(case, seed):
    rng, gen = random.Random(seed), _gen(seed)
    s = {"case": case}
    if case["op"] == "plan":
        _prepare_plan(case, rng, gen, s)
    elif case["op"] == "verify":
        _prepare_verify(case, rng, gen, s)
    else:
        H, d, gs, rk, rv = SHAPES[case["shape"]]
        G, W = H // gs, gs * d
        lens = _lens(case, rng, case.get("queries", 1))
        s["table"], s["pages"] = _tables(lens, case["context"], gen)
        s["lens"] = _ints(lens)
        explicit = case.get("explicit", False)
        s["pos_pool"] = _positions(lens, s["table"], s["pages"], explicit)
        if case["op"] == "bounds":
            s["zk"], s["zks"] = _pool(s["pages"], G, rk, case["lat"], gen)
            s["Bk"] = _factor(G, rk, W, case["act"], gen)
            s["first"] = _ints([max(0, (-(-t // PAGE) - case["span"]) * PAGE) for t in lens])
            # one page more than the cache has: where the plain form puts what it must not write
            s["bounds"] = torch.zeros((s["pages"] + 1, G, 2, W), dtype=TYPES[case["act"]], device="cuda")
        else:
            Q = case["queries"]
            s["q"] = torch.randn((len(lens), Q, H, d), generator=gen, device="cuda").to(TYPES[case["act"]])
            at = [[max(0, t - Q + j) for j in range(Q)] for t in lens]
            s["q_pos"] = _ints([[3 * p + 1 if explicit else p for p in row] for row in at])
            # pages that hold a token at or before the query (a single query sees every page)
            seen = [[-(-min(t, p + 1) // PAGE) for p in row] for t, row in zip(lens, at)]
            if case["op"] == "select":
                mid = torch.randn((s["pages"], G, W), generator=gen, device="cuda") * 0.6
                half = torch.rand((s["pages"], G, W), generator=gen, device="cuda") + 1.9
                s["bounds"] = torch.stack([mid - half, mid + half], 2).to(TYPES[case["act"]])
                s["list"] = torch.empty((len(lens), Q, G, case["keep"]), dtype=torch.int32, device="cuda")
                s["counts"] = torch.empty((len(lens), Q, G), dtype=torch.int32, device="cuda")
                s["scores"] = torch.empty((len(lens), Q, G, case["keep"]), device="cuda")
            else:
                s["zk"], s["zks"] = _pool(s["pages"], G, rk, case["lat"], gen)
                s["zv"], s["zvs"] = _pool(s["pages"], G, rv, case["lat"], gen)
                s["Bk"], s["Bv"] = _factor(G, rk, W, case["act"], gen), _factor(G, rv, W, case["act"], gen)
                s["list"], s["counts"] = _some_pages(_ints(seen), s["table"].shape[1], G, case["keep"], gen)
                s["out"] = torch.empty_like(s["q"])
                s["lse"] = torch.empty((len(lens), Q, H), dtype=torch.float32, device="cuda")
    if own:
        _handles(s)
    return s


def _some_pages(seen, wide, G, keep, gen):
    """For each query and group `keep` of its pages (all where it has fewer), ascending, the last among them."""
    batch, Q = seen.shape
    score = torch.rand((batch, Q, G, wide), generator=gen, device="cuda")
    page = torch.arange(wide, device="cuda")
    last = seen.view(batch, Q, 1, 1) - 1
    score = torch.where(page == last, 2.0, torch.where(page < last, score, -1.0))
    top = torch.topk(score, min(keep, wide), dim=-1)
    ids = torch.where(top.values >= 0, top.indices, wide).sort(-1).values
    ids = torch.nn.functional.pad(torch.where(ids < wide, ids, -1), (0, keep - ids.shape[-1]), value=-1)
    return ids.to(torch.int32).contiguous(), (ids >= 0).sum(-1).to(torch.int32)


def _prepare_plan(case, rng, gen, s):
    """A server's page state in one buffer, and what each request appends (or drops, when it is finished)."""
    B, decode = case["batch"], case["kind"] == "decode"
    lens = [rng.randint(0 if not decode else 1, case["context"]) for _ in range(B)]
    leaves = [] if decode else rng.sample(range(B), B // 7)
    stay = [i for i in range(B) if i not in leaves]
    new = [1] * B
    if not decode:
        share = [rng.uniform(0.2, 1.8) for _ in stay]
        cuts = [int(case["tokens"] * sum(share[:k]) / sum(share)) for k in range(len(stay))] + [case["tokens"]]
        for k, i in enumerate(stay):
            new[i] = cuts[k + 1] - cuts[k]
        for i in leaves:
            new[i] = -lens[i] if rng.random() < 0.7 else -rng.randint(0, lens[i])
    used = [-(-t // PAGE) for t in lens]
    need = sum(max(0, -(-(t + n) // PAGE) - u) for t, n, u in zip(lens, new, used))
    # the pool holds the longest lengths, a row of the page table the largest share of the new tokens
    total = B * -(-case["context"] // PAGE) + case["tokens"] // PAGE + B + 9
    wide = -(-(case["context"] + (1 if decode else min(case["tokens"], 9 * case["tokens"] // len(stay) + 1))) // PAGE)
    free = total - sum(used) if rng.random() < 0.8 else (3 * need) // 4        # now and then too few
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = total - sum(used)
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    # [seq_lens | num_free | free stack | page table], as the server keeps it and as it was before the step
    stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    stack[:free] = order[:free]
    s["before"] = torch.cat([_ints(lens), _ints([free]), stack, table.reshape(-1)])
    s["now"] = s["before"].clone()
    s["cut"] = (B, total, wide)
    s["new"] = _ints(new)
    rows = case["tokens"] + case["spare"]           # a padded batch has rows that no request owns
    s["slots"], s["positions"] = _ints([0] * rows), _ints([0] * rows)
    s["starts"], s["taken"] = _ints([0] * (B + 1)), _ints([0] * B)


def _plan_views(s, buf):
    B, total, wide = s["cut"]
    lens, free, stack, table = torch.split(buf, [B, 1, total, B * wide])
    return lens, free, stack, table.view(B, wide)


def _prepare_verify(case, rng, gen, s):
    """Target and draft distributions that lie near each other, drafts sampled from the draft's."""
    B, D, V, dt = case["batch"], case["drafts"], case["vocab"], TYPES[case["dtype"]]
    wide = V + case["pad"]
    logits = torch.randn((B, D + 1, V), generator=gen, device="cuda") * 2.5
    target = torch.zeros((B, D + 1, wide), dtype=dt, device="cuda")
    target[..., :V] = torch.softmax(logits, -1).to(dt)
    near = logits[:, :D] + 0.4 * torch.randn((B, D, V), generator=gen, device="cuda")
    noise = torch.empty((B, D, V), device="cuda").exponential_(generator=gen)
    s["drafts"] = (torch.softmax(near, -1) / noise).argmax(-1).to(torch.int32)
    s["target"], s["draft"] = target[..., :V], None
    if case["drafter"] == "probs":
        draft = torch.zeros((B, D, wide), dtype=dt, device="cuda")
        draft[..., :V] = torch.softmax(near, -1).to(dt)
        s["draft"] = draft[..., :V]
    s["draft_lens"] = _ints([rng.choice([D, D, rng.randint(0, D)]) for _ in range(B)])
    s["u_accept"] = torch.rand((B, D), generator=gen, device="cuda")
    s["u_sample"] = torch.rand((B,), generator=gen, device="cuda")
    s["tokens"] = torch.empty((B, D + 1), dtype=torch.int32, device="cuda")
    s["accepted"], s["rollback"] = _ints([0] * B), _ints([0] * B)


def _handles(s):
    """The config and the workspace that a user of the framework keeps."""
    from rank_kv_cache_palu_b200 import api as P
    c = s["case"]
    if c["op"] == "plan":
        n = P.palu_plan_workspace_size(c["batch"])
    elif c["op"] == "verify":
        n = P.palu_verify_workspace_size(c["batch"], c["drafts"], c["vocab"])
    else:
        H, d, gs, rk, rv = SHAPES[c["shape"]]
        s["cfg"] = cfg = P.make_config(H, d, gs, rk, rv, PAGE, c["rope"], c["act"], c.get("lat"))
        wide = s["table"].shape[1]
        if c["op"] == "bounds":
            n = P.palu_page_bounds_workspace_size(cfg, c["batch"], wide)
        elif c["op"] == "select":
            n = P.palu_select_workspace_size(cfg, c["batch"], c["queries"], wide)
        else:
            n = P.palu_decode_pages_workspace_size(cfg, c["batch"], c["queries"], c["keep"])
    s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ a pass
def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state)


def _run_own(op, s):
    from rank_kv_cache_palu_b200 import api as P
    if op == "plan":
        s["now"].copy_(s["before"])
        lens, free, stack, table = _plan_views(s, s["now"])
        P.palu_plan_append(PAGE, s["new"], lens, table, stack, free, s["slots"], s["positions"], s["starts"],
                           s["taken"], s["ws"])
        return {"slots": s["slots"], "positions": s["positions"], "starts": s["starts"], "taken": s["taken"],
                "lens": lens, "free": free, "stack": stack, "table": table}
    if op == "verify":
        P.palu_verify_drafts(s["target"], s["draft"], s["drafts"], s["draft_lens"], s["u_accept"], s["u_sample"],
                             s["tokens"], s["accepted"], s["rollback"], s["ws"])
        return {"tokens": s["tokens"], "accepted": s["accepted"], "rollback": s["rollback"]}
    if op == "bounds":
        P.palu_page_bounds(s["cfg"], s["first"], s["zk"], s["zks"], s["pos_pool"], s["table"], s["lens"],
                           s["pages"], s["Bk"], s["bounds"][:s["pages"]], s["ws"])
        return s["bounds"][:s["pages"]]
    if op == "select":
        P.palu_select_pages(s["cfg"], s["q"], s["q_pos"], s["bounds"], s["pos_pool"], s["table"], s["lens"],
                            s["pages"], 1, 2, s["list"], s["counts"], s["scores"], s["ws"])
        return {"list": s["list"], "counts": s["counts"], "scores": s["scores"]}
    P.palu_decode_attn_pages(s["cfg"], s["q"], s["q_pos"], s["zk"], s["zv"], s["zks"], s["zvs"], s["pos_pool"],
                             s["table"], s["lens"], s["list"], s["counts"], s["pages"], s["Bk"], s["Bv"], s["out"],
                             s["lse"], s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _run_plain(op, s):
    return {"plan": _plain_plan, "verify": _plain_verify, "bounds": _plain_bounds, "select": _plain_select,
            "attend": _plain_attend}[op](s)


def _plain_plan(s):
    B, total, wide = s["cut"]
    lens, free, stack, table = (v.long() for v in _plan_views(s, s["before"]))
    new, rows = s["new"].long(), s["slots"].shape[0]
    starts = torch.nn.functional.pad(new.clamp(min=0).cumsum(0), (1, 0))
    left = lens + new
    good = (left >= 0) & (left <= wide * PAGE) & (starts[1:] <= rows)
    new = torch.where(good, new, 0)
    had = (lens + PAGE - 1) // PAGE
    need = ((lens + new + PAGE - 1) // PAGE - had).clamp(min=0)
    through = need.cumsum(0)
    fits = (need == 0) | (through <= free)
    new, need = torch.where(fits, new, 0), torch.where(fits, need, 0)
    before = need.cumsum(0) - need
    got = need.sum()
    has = (lens + new + PAGE - 1) // PAGE
    # rows
    row = torch.arange(rows, device=lens.device)
    b = torch.searchsorted(starts[1:].contiguous(), row, right=True).clamp(max=B - 1)
    live = (row < starts[-1]) & (new[b] > 0)
    pos = torch.where(live, lens[b] + row - starts[b], 0)
    lp = pos // PAGE
    fresh = lp >= had[b]
    page = torch.where(fresh, stack[(free - 1 - (before[b] + lp - had[b])).clamp(0, total - 1)],
                       table[b, lp.clamp(max=wide - 1)])
    slots = torch.where(live, page * PAGE + pos % PAGE, -1)
    # page table, then the pages given back: the first of them in (request, page) order ends on top
    table = torch.nn.functional.pad(table, (0, 1))
    table[b, torch.where(live & fresh, lp, wide)] = page
    table = table[:, :wide].contiguous()
    col = torch.arange(wide, device=lens.device)
    gone = (col >= has[:, None]) & (col < had[:, None])
    back = gone.sum()
    rank = gone.reshape(-1).cumsum(0).view(B, wide) - 1
    stack = torch.nn.functional.pad(stack, (0, 1))
    stack[torch.where(gone, free - got + back - 1 - rank, total)] = table
    table = torch.where(gone, -1, table)
    out = {"slots": slots, "positions": pos, "starts": starts, "taken": new, "lens": lens + new,
           "free": free - got + back, "stack": stack[:total], "table": table}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_verify(s):
    D = s["case"]["drafts"]
    x, n = s["drafts"].long(), s["draft_lens"].long()
    p_x = s["target"][:, :D].gather(-1, x[..., None])[..., 0].double()
    q_x = s["draft"].gather(-1, x[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p_x)
    i = torch.arange(D + 1, device=x.device)
    yes = (s["u_accept"].double() * q_x < p_x) & (i[:D] < n[:, None])
    a = yes.long().cumprod(-1).sum(-1)
    row = torch.arange(x.shape[0], device=x.device)
    p = s["target"][row, a].double()
    at = a.clamp(max=D - 1)
    if s["draft"] is not None:
        q = s["draft"][row, at].double()
    else:
        q = (torch.arange(p.shape[-1], device=x.device) == x[row, at][:, None]).double()
    w = (p - torch.where((a < n)[:, None], q, 0.0)).clamp(min=0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    c = w.cumsum(-1)
    token = (c <= s["u_sample"].double()[:, None] * c[:, -1:]).sum(-1)
    padded = torch.nn.functional.pad(x, (0, 1))
    tokens = torch.where(i < a[:, None], padded, torch.where(i == a[:, None], token[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "accepted": a.to(torch.int32), "rollback": (a - n).to(torch.int32)}


def _rotate(v, pos, base):
    """Rotate-half RoPE of v [..., d] at pos [...], the angles in 64 bits."""
    if not base:
        return v
    half = v.shape[-1] // 2
    freq = base ** (-2.0 * torch.arange(half, device=v.device, dtype=torch.float64) / v.shape[-1])
    angle = pos.double()[..., None] * freq
    cos, sin = angle.cos().to(v.dtype), angle.sin().to(v.dtype)
    a, b = v[..., :half], v[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _latents(pool, scales, page, groups, group, rank, lat, act):
    """Latents [..., PAGE, rank] of (page, group), both [...], in 32 bits: the swizzle undone, codes scaled."""
    size = {"f32": 4, "f16": 2, "bf16": 2, "int4": 0}[lat]
    kind = TYPES[lat] if size else torch.uint8
    per = 16 // size if size else 16                         # entries (int4: bytes) per 16-byte unit
    blocks = pool.view(kind).view(-1, (rank if size else rank // 2) // (8 * per), PAGE, 8, per)
    which = page * groups + group
    token = torch.arange(PAGE, device=pool.device)[:, None]
    z = blocks[which][..., token, torch.arange(8, device=pool.device) ^ (token % 8), :]   # [..., nb, PAGE, 8, per]
    z = z.movedim(-4, -3).flatten(-3)
    if size:
        return z.float()
    code = torch.stack([z & 15, z >> 4], -1).flatten(-2).to(torch.int8)
    code = torch.where(code > 7, code - 16, code).float()
    scale = scales.view(torch.float16).view(-1, PAGE, scales.numel() // 2 // (blocks.shape[0] * PAGE))[which]
    scale = scale[..., :rank // 32].float().repeat_interleave(32, -1)
    return (code * scale).to(TYPES[act]).float()


def _outwards(v, dtype, up):
    """v in the type, rounded up or down."""
    if dtype == torch.float32:
        return v
    r = v.to(dtype)
    bits = r.view(torch.int16)
    step = torch.where(bits >= 0, 1, -1) * (1 if up else -1)
    away = torch.where(r == 0, torch.tensor(1 if up else -32767, dtype=torch.int16, device=v.device),
                       (bits + step).to(torch.int16)).view(dtype)
    return torch.where(r.float() < v if up else r.float() > v, away, r)


def _plain_bounds(s):
    c = s["case"]
    H, d, gs, rk, _ = SHAPES[c["shape"]]
    G, base = H // gs, c["rope"]
    lens = s["lens"].long()
    lp = s["first"].long()[:, None] // PAGE + torch.arange(c["span"], device=lens.device)
    live = lp * PAGE < lens[:, None]
    page = torch.where(live, s["table"].long().gather(1, lp.clamp(max=s["table"].shape[1] - 1)), 0)
    z = _latents(s["zk"], s["zks"], page[..., None], G, torch.arange(G, device=lens.device), rk, c["lat"], c["act"])
    k = (z @ s["Bk"].float()).view(*z.shape[:-1], gs, d)     # [b, span, G, PAGE, gs, d]
    t = lp[..., None] * PAGE + torch.arange(PAGE, device=lens.device)
    pos = t if s["pos_pool"] is None else s["pos_pool"][page]
    k = _rotate(k, pos[:, :, None, :, None], base)
    dead = (t >= lens[:, None, None])[:, :, None, :, None, None]
    lo = k.masked_fill(dead, math.inf).amin(3).flatten(-2)
    hi = k.masked_fill(dead, -math.inf).amax(3).flatten(-2)
    kind = TYPES[c["act"]]
    s["bounds"][torch.where(live, page, s["pages"])] = torch.stack([_outwards(lo, kind, False), _outwards(hi, kind, True)], 3)
    return s["bounds"][:s["pages"]]


def _visible(s):
    """Tokens each query of the step may see: all of the sequence for one query, else those up to its own."""
    T = s["lens"].long()[:, None]
    if s["case"]["queries"] == 1 or s["pos_pool"] is not None:
        return T.expand(-1, s["case"]["queries"])
    return torch.minimum(T, s["q_pos"].long() + 1)


def _plain_select(s):
    c = s["case"]
    H, d, gs, _, _ = SHAPES[c["shape"]]
    G, Q, keep = H // gs, c["queries"], c["keep"]
    q = _rotate(s["q"].double(), s["q_pos"][..., None], c["rope"])      # 64 bits: pages next to the border
    q = q.view(q.shape[0], Q, G, gs, d)
    bounds = s["bounds"][s["table"].long().clamp(min=0)].double()         # [b, n, G, 2, W]
    n = bounds.shape[1]
    lo, hi = bounds.view(*bounds.shape[:4], gs, d).unbind(3)
    up = torch.einsum("bqghd,bnghd->bqghn", q.clamp(min=0), hi) + torch.einsum("bqghd,bnghd->bqghn", q.clamp(max=0), lo)
    score = up.amax(3)
    seen = ((_visible(s) + PAGE - 1) // PAGE)[:, :, None, None]
    page = torch.arange(n, device=q.device)
    first = torch.where((page < 1) | (page >= seen - 2), math.inf, score)
    first = torch.where(page < seen, first, -math.inf)
    top = first.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    ids = torch.where(top < seen, top, n).sort(-1).values
    count = (ids < n).sum(-1)
    kept = torch.where(ids < n, score.gather(-1, ids.clamp(max=n - 1)), -math.inf)
    pad = (0, keep - ids.shape[-1])
    ids = torch.nn.functional.pad(torch.where(ids < n, ids, -1), pad, value=-1)
    kept = torch.nn.functional.pad(kept, pad, value=-math.inf)
    return {"list": ids.to(torch.int32), "counts": count.to(torch.int32), "scores": kept.float()}


def _plain_attend(s):
    c = s["case"]
    H, d, gs, rk, rv = SHAPES[c["shape"]]
    G, Q, base, kind = H // gs, c["queries"], c["rope"], TYPES[c["act"]]
    B, lp = s["lens"].shape[0], s["list"].long()             # [b, Q, G, K]
    K, live = lp.shape[-1], lp >= 0
    row = torch.arange(B, device=lp.device)[:, None, None, None]
    page = torch.where(live, s["table"].long()[row, lp.clamp(min=0)], 0)
    group = torch.arange(G, device=lp.device)[:, None].expand(G, K)
    zk = _latents(s["zk"], s["zks"], page, G, group, rk, c["lat"], c["act"]).flatten(3, 4)      # [b, Q, G, K·PAGE, r]
    t = lp[..., None] * PAGE + torch.arange(PAGE, device=lp.device)
    pos = t if s["pos_pool"] is None else s["pos_pool"][page].long()
    dead = ~live[..., None] | (t >= s["lens"].long()[:, None, None, None, None])
    if Q > 1:
        dead = dead | (pos > s["q_pos"].long()[:, :, None, None, None])
    k = (zk @ s["Bk"].float()).view(B, Q, G, K * PAGE, gs, d)
    k = _rotate(k, pos.reshape(B, Q, G, K * PAGE, 1), base)
    q = _rotate(s["q"].float(), s["q_pos"][..., None], base).view(B, Q, G, 1, gs, d)
    score = (k * q).sum(-1) / math.sqrt(d)                    # [b, Q, G, K·PAGE, gs]
    del k, zk
    score = score.masked_fill(dead.view(B, Q, G, K * PAGE, 1), -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    zv = _latents(s["zv"], s["zvs"], page, G, group, rv, c["lat"], c["act"]).flatten(3, 4)
    zv = zv.masked_fill(dead.view(B, Q, G, K * PAGE, 1), 0.0)
    a = (p / torch.where(total == 0, 1.0, total)).transpose(3, 4) @ zv                           # [b, Q, G, gs, r_v]
    Bv = s["Bv"].float().view(G, rv, gs, d).transpose(1, 2)
    out = (a[..., None, :] @ Bv).view(B, Q, H, d)
    lse = (top + total.log()).view(B, Q, H)
    return {"out": out.to(kind), "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        B, n = case["batch"], case["tokens"]
        # lengths and changes in, row starts, lengths and changes out; slots and positions; new pages in and out
        return {"bytes": 4.0 * (5 * B + 2 * n + 3 * (n / PAGE)), "flops": 0.0}
    size = {"f32": 4, "f16": 2, "bf16": 2}[case.get("dtype") or case["act"]]
    if case["op"] == "verify":
        # the row that the sample is taken from, of the target and of the draft
        rows = 2 if case["drafter"] == "probs" else 1
        return {"bytes": float(case["batch"] * (rows * case["vocab"] * size + 8 * case["drafts"])),
                "flops": 3.0 * case["batch"] * case["vocab"]}
    H, d, gs, rk, rv = SHAPES[case["shape"]]
    G, W, B = H // gs, gs * d, case["batch"]
    if case["op"] == "select":
        pages = B * min(-(-case["context"] // PAGE), 1 << 30)
        return {"bytes": float(pages * G * 2 * W * size), "flops": 2.0 * pages * G * W * case["queries"]}
    row = {"int4": 0.5 + 2 / 32}.get(case["lat"], size)
    if case["op"] == "bounds":
        pages = B * min(case["span"], -(-case["context"] // PAGE))
        return {"bytes": G * (pages * (PAGE * rk * row + 2 * W * size) + rk * W * size),
                "flops": 2.0 * pages * PAGE * G * rk * W}
    tokens = B * case["queries"] * min(case["keep"] * PAGE, case["context"])
    return {"bytes": G * (tokens * (rk + rv) * row + (rk + rv) * W * size),
            "flops": tokens * G * (2.0 * rk * W if case["rope"] else 2.0 * gs * rk) + tokens * G * 2.0 * gs * rv}


# ------------------------------------------------------------------ the definition in 64 bits
def _bytes_of(case, pool, scales, page, group, groups, rank):
    """Latents [PAGE, rank] of one block in 64 bits, each entry fetched from its own place: entry e of token t
    lies in column block o // 128 of the block, o its byte, its 16-byte unit XORed with t mod 8."""
    lat, act = case["lat"], TYPES[case["act"]]
    t = torch.arange(PAGE, device=pool.device)[:, None]
    e = torch.arange(rank, device=pool.device)[None, :]
    if lat == "int4":
        o, row = e // 2, rank // 2
    else:
        row = rank * TYPES[lat].itemsize
        o = e * TYPES[lat].itemsize
    at = (page * groups + group) * PAGE * row + (o // 128) * PAGE * 128 + t * 128 + (((o % 128) // 16) ^ (t % 8)) * 16 + o % 16
    if lat != "int4":
        return pool.view(TYPES[lat])[at // TYPES[lat].itemsize].double()
    nibble = (pool[at].long() >> (4 * (e % 2))) & 15
    code = (nibble + 8) % 16 - 8
    srow = -(-2 * (rank // 32) // 16) * 8
    scale = scales.view(torch.float16)[((page * groups + group) * PAGE + t) * srow + e // 32]
    return (code * scale.double()).to(act).double()


def _turn(v, pos, base):
    """RoPE as a product of complex numbers, in 64 bits."""
    if base == 0:
        return v
    n = v.shape[-1] // 2
    w = torch.exp(-2 * math.log(base) / v.shape[-1] * torch.arange(n, device=v.device, dtype=torch.float64))
    ang = pos.double().unsqueeze(-1) * w
    z = torch.complex(v[..., :n].contiguous(), v[..., n:].contiguous()) * torch.complex(ang.cos(), ang.sin())
    return torch.cat([z.real, z.imag], -1)


def _exact_scores(case, s, lens, table, G, gs, d):
    """The bounds of the pages that are kept, from the definition: the larger of q lo and q hi, summed."""
    Q, keep = case["queries"], case["keep"]
    out = torch.full((len(lens), Q, G, keep), -math.inf, dtype=torch.float64, device="cuda")
    for i, t in enumerate(lens):
        for j, at in enumerate(s["q_pos"][i].tolist()):
            n = -(-(t if Q == 1 else min(t, at + 1)) // PAGE)
            if n == 0:
                continue
            q = _turn(s["q"][i, j].double(), s["q_pos"][i, j], case["rope"]).view(1, G, 1, gs, d)
            box = s["bounds"][torch.tensor(table[i][:n], device="cuda")].double().view(n, G, 2, gs, d)
            score = (q * box).max(2).values.sum(-1).max(-1).values.T        # [G, n]
            order = score.clone()
            order[:, :1] = order[:, max(0, n - 2):] = math.inf
            kept = torch.argsort(order, dim=1, descending=True, stable=True)[:, :keep].sort(1).values
            out[i, j, :, :kept.shape[1]] = score.gather(1, kept)
    return out


def exact(case, seed):
    if case["op"] in ("plan", "verify"):
        return None                                           # whole numbers only
    s = prepare(case, seed)
    H, d, gs, rk, rv = SHAPES[case["shape"]]
    G = H // gs
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if case["op"] == "select":
        return {"list": None, "counts": None, "scores": _exact_scores(case, s, lens, table, G, gs, d)}
    Bk = s["Bk"].double()

    def keys(i, lp, g):
        n = min(PAGE, lens[i] - lp * PAGE)
        page = table[i][lp]
        z = _bytes_of(case, s["zk"], s["zks"], page, g, G, rk)[:n]
        at = torch.arange(lp * PAGE, lp * PAGE + n, device=z.device) if s["pos_pool"] is None else s["pos_pool"][page, :n]
        return _turn((z @ Bk[g]).view(n, gs, d), at[:, None], case["rope"]), at, page, n

    if case["op"] == "bounds":
        out = torch.zeros((s["pages"], G, 2, gs * d), dtype=torch.float64, device="cuda")
        for i, first in enumerate(s["first"].tolist()):
            for lp in range(first // PAGE, -(-lens[i] // PAGE)):
                for g in range(G):
                    k, _, page, n = keys(i, lp, g)
                    out[page, g, 0], out[page, g, 1] = k.view(n, -1).min(0).values, k.view(n, -1).max(0).values
        return out
    if case["batch"] * case["queries"] * G * case["keep"] > 20000:
        return None
    Q = case["queries"]
    out = torch.zeros((len(lens), Q, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), Q, H), -math.inf, dtype=torch.float64, device="cuda")
    lists, q_pos = s["list"].tolist(), s["q_pos"].tolist()
    Bv = s["Bv"].double()
    for i in range(len(lens)):
        for j in range(Q):
            q = _turn(s["q"][i, j].double(), s["q_pos"][i, j], case["rope"])
            for g in range(G):
                scores, values = [], []
                for lp in lists[i][j][g]:
                    if lp < 0:
                        continue
                    k, at, page, n = keys(i, lp, g)
                    sc = (k * q[g * gs:(g + 1) * gs]).sum(-1).T / d ** 0.5
                    if Q > 1:
                        sc[:, at > q_pos[i][j]] = -math.inf
                    scores.append(sc)
                    values.append(_bytes_of(case, s["zv"], s["zvs"], page, g, G, rv)[:n])
                if not scores:
                    continue
                sc = torch.cat(scores, 1)
                total = torch.logsumexp(sc, 1)
                p = torch.where(total[:, None] == -math.inf, 0.0, torch.exp(sc - total[:, None]))
                v = torch.cat(values) @ Bv[g]
                for h in range(gs):
                    out[i, j, g * gs + h] = p[h] @ v[:, h * d:(h + 1) * d]
                lse[i, j, g * gs:(g + 1) * gs] = total
    return {"out": out, "lse": lse}
