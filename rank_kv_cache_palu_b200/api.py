"""Python binding of libpalu.so: the C-ABI entry points under the same names.

Argument marshalling only — every step of the path runs in the CUDA kernels.
Tensors are torch tensors used as device buffers; streams are torch streams.
Each call raises ``PaluError`` when the library returns a non-OK status.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple

import torch

from ._lib import PaluConfig, load

DTYPE_CODE = {"f32": 0, "f16": 1, "bf16": 2, "int4": 3}
TORCH_OF = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

STATUS_NAMES = {
    0: "PALU_OK", 1: "PALU_ERR_INVALID_ARG", 2: "PALU_ERR_UNSUPPORTED", 3: "PALU_ERR_ALIGNMENT",
    4: "PALU_ERR_WORKSPACE", 5: "PALU_ERR_CUDA", 6: "PALU_ERR_DEVICE_TIMEOUT",
    7: "PALU_ERR_DEVICE_BOUNDS",
}


class PaluError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.palu_status_string(status).decode()
        if status == 5:
            msg += f" ({lib.palu_last_cuda_error().decode()})"
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise PaluError(status, where)


def make_config(num_heads: int, head_dim: int, group_size: int, rank_k: int, rank_v: int,
                page_size: int = 128, rope_base: float = 10000.0, act_dtype: str = "bf16",
                latent_dtype: str | None = None) -> PaluConfig:
    return PaluConfig(num_heads, head_dim, group_size, rank_k, rank_v, page_size, float(rope_base),
                      DTYPE_CODE[act_dtype], DTYPE_CODE[latent_dtype or act_dtype])


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if t.numel() > 0 and not t.is_cuda:
        raise ValueError("palu tensors must live in CUDA device memory")
    if not t.is_contiguous():
        raise ValueError("palu tensors must be contiguous")
    return t.data_ptr() if t.numel() > 0 else None


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def palu_cache_strides(cfg: PaluConfig) -> tuple[int, int, int, int]:
    out = [ctypes.c_size_t() for _ in range(4)]
    _check(load().palu_cache_strides(ctypes.byref(cfg), *[ctypes.byref(o) for o in out]),
           "palu_cache_strides")
    return tuple(o.value for o in out)


def palu_compress_workspace_size(cfg: PaluConfig, n_tokens: int, d_model: int) -> int:
    out = ctypes.c_size_t()
    _check(load().palu_compress_workspace_size(ctypes.byref(cfg), n_tokens, d_model,
                                               ctypes.byref(out)), "palu_compress_workspace_size")
    return out.value


def palu_decode_num_splits(cfg: PaluConfig, batch: int, max_pages: int) -> int:
    out = ctypes.c_int()
    _check(load().palu_decode_num_splits(ctypes.byref(cfg), batch, max_pages, ctypes.byref(out)),
           "palu_decode_num_splits")
    return out.value


def palu_decode_workspace_size(cfg: PaluConfig, batch: int, max_pages: int, num_splits: int = 0) -> int:
    out = ctypes.c_size_t()
    _check(load().palu_decode_workspace_size(ctypes.byref(cfg), batch, max_pages, num_splits,
                                             ctypes.byref(out)), "palu_decode_workspace_size")
    return out.value


def palu_decode_kernel_kind(cfg: PaluConfig) -> int:
    return int(load().palu_decode_kernel_kind(ctypes.byref(cfg)))


def palu_kernel_launches() -> int:
    """Kernels launched by libpalu in this process so far."""
    return int(load().palu_kernel_launches())


def palu_debug_trace(buffer, tiles_per_cta: int = 0) -> None:
    """Record tensor-core decode phase timestamps into `buffer` (int64 CUDA tensor); None stops."""
    if buffer is None:
        _check(load().palu_debug_trace(None, 0, 0), "palu_debug_trace")
    else:
        _check(load().palu_debug_trace(_ptr(buffer), buffer.numel() * buffer.element_size(),
                                       tiles_per_cta), "palu_debug_trace")


def palu_debug_timeout_test(wait_cycles: int = 0, stall: bool = False) -> None:
    """Test hook of the kernels' timeout path: bound every wait of later tensor-core
    launches to wait_cycles SM cycles (0 = the default) and, with stall, make each
    such launch run that bound out.  palu_debug_timeout_test() restores normal operation."""
    _check(load().palu_debug_timeout_test(int(wait_cycles), 1 if stall else 0), "palu_debug_timeout_test")


def palu_compress_append(cfg: PaluConfig, x, A_k, A_v, slot_mapping, positions, zk_pool, zv_pool,
                         zk_scales, zv_scales, pos_pool, num_pages: int, workspace, stream=None):
    n, d_model = x.shape
    st = load().palu_compress_append(
        ctypes.byref(cfg), n, d_model, _ptr(x), _ptr(A_k), _ptr(A_v), _ptr(slot_mapping),
        _ptr(positions), _ptr(zk_pool), _ptr(zv_pool), _ptr(zk_scales), _ptr(zv_scales),
        _ptr(pos_pool), num_pages, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "palu_compress_append")


def palu_decode_attn(cfg: PaluConfig, q, q_pos, zk_pool, zv_pool, zk_scales, zv_scales, pos_pool,
                     page_table, seq_lens, num_pages: int, B_k, B_v, out, lse, workspace,
                     num_splits: int = 0, stream=None):
    batch = q.shape[0]
    max_pages = page_table.shape[1]
    st = load().palu_decode_attn(
        ctypes.byref(cfg), batch, _ptr(q), _ptr(q_pos), _ptr(zk_pool), _ptr(zv_pool),
        _ptr(zk_scales), _ptr(zv_scales), _ptr(pos_pool), _ptr(page_table), max_pages,
        _ptr(seq_lens), num_pages, _ptr(B_k), _ptr(B_v), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), num_splits, _stream(stream))
    _check(st, "palu_decode_attn")


MAX_QUERIES = 16


def palu_decode_multi_workspace_size(cfg: PaluConfig, batch: int, num_queries: int, max_pages: int,
                                     num_splits: int = 0) -> int:
    out = ctypes.c_size_t()
    _check(load().palu_decode_multi_workspace_size(ctypes.byref(cfg), batch, num_queries, max_pages,
                                                   num_splits, ctypes.byref(out)),
           "palu_decode_multi_workspace_size")
    return int(out.value)


def palu_decode_attn_multi(cfg: PaluConfig, q, q_pos, zk_pool, zv_pool, zk_scales, zv_scales, pos_pool,
                           page_table, seq_lens, num_pages: int, B_k, B_v, out, lse, workspace,
                           num_splits: int = 0, stream=None):
    """Several query tokens per sequence: q [batch][Q][H][d_h], q_pos [batch][Q]; causal by position."""
    batch, nq = q.shape[0], q.shape[1]
    max_pages = page_table.shape[1]
    st = load().palu_decode_attn_multi(
        ctypes.byref(cfg), batch, nq, _ptr(q), _ptr(q_pos), _ptr(zk_pool), _ptr(zv_pool),
        _ptr(zk_scales), _ptr(zv_scales), _ptr(pos_pool), _ptr(page_table), max_pages,
        _ptr(seq_lens), num_pages, _ptr(B_k), _ptr(B_v), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), num_splits, _stream(stream))
    _check(st, "palu_decode_attn_multi")


def _ranks(r):
    """Host int32 array of per-group ranks (None: the config's uniform ranks)."""
    return None if r is None else (ctypes.c_int32 * len(r))(*[int(v) for v in r])


def palu_cache_strides_ranked(cfg: PaluConfig, ranks_k, ranks_v):
    """(k_page, v_page, k_scale_page, v_scale_page, k_group_offsets, v_group_offsets) in bytes."""
    G = cfg.num_heads // cfg.group_size
    out = [ctypes.c_size_t() for _ in range(4)]
    ko, vo = (ctypes.c_size_t * G)(), (ctypes.c_size_t * G)()
    _check(load().palu_cache_strides_ranked(ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v),
                                            *[ctypes.byref(o) for o in out], ko, vo),
           "palu_cache_strides_ranked")
    return (*[o.value for o in out], list(ko), list(vo))


def palu_compress_ranked_workspace_size(cfg: PaluConfig, ranks_k, ranks_v, n_tokens: int, d_model: int) -> int:
    out = ctypes.c_size_t()
    _check(load().palu_compress_ranked_workspace_size(ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v),
                                                      n_tokens, d_model, ctypes.byref(out)),
           "palu_compress_ranked_workspace_size")
    return int(out.value)


def palu_compress_append_ranked(cfg: PaluConfig, ranks_k, ranks_v, x, A_k, A_v, slot_mapping, positions,
                                zk_pool, zv_pool, zk_scales, zv_scales, pos_pool, num_pages: int, workspace,
                                stream=None):
    """palu_compress_append for a layer with a rank pair per group (A columns stacked by group)."""
    n, d_model = x.shape
    st = load().palu_compress_append_ranked(
        ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v), n, d_model, _ptr(x), _ptr(A_k), _ptr(A_v),
        _ptr(slot_mapping), _ptr(positions), _ptr(zk_pool), _ptr(zv_pool), _ptr(zk_scales), _ptr(zv_scales),
        _ptr(pos_pool), num_pages, _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream))
    _check(st, "palu_compress_append_ranked")


def palu_decode_ranked_workspace_size(cfg: PaluConfig, ranks_k, ranks_v, batch: int, num_queries: int,
                                      max_pages: int, num_splits: int = 0) -> int:
    out = ctypes.c_size_t()
    _check(load().palu_decode_ranked_workspace_size(ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v), batch,
                                                    num_queries, max_pages, num_splits, ctypes.byref(out)),
           "palu_decode_ranked_workspace_size")
    return int(out.value)


def palu_decode_attn_ranked(cfg: PaluConfig, ranks_k, ranks_v, q, q_pos, zk_pool, zv_pool, zk_scales, zv_scales,
                            pos_pool, page_table, seq_lens, num_pages: int, B_k, B_v, out, lse, workspace,
                            num_splits: int = 0, stream=None):
    """Decode step of a layer with a rank pair per group: q [batch][Q][H][d_h], q_pos [batch][Q]
    (Q = 1 is the single-query step); B_k / B_v rows stacked by group."""
    batch, nq = q.shape[0], q.shape[1]
    max_pages = page_table.shape[1]
    st = load().palu_decode_attn_ranked(
        ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v), batch, nq, _ptr(q), _ptr(q_pos), _ptr(zk_pool),
        _ptr(zv_pool), _ptr(zk_scales), _ptr(zv_scales), _ptr(pos_pool), _ptr(page_table), max_pages,
        _ptr(seq_lens), num_pages, _ptr(B_k), _ptr(B_v), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), num_splits, _stream(stream))
    _check(st, "palu_decode_attn_ranked")


NOALLOC_SCRATCH_BYTES = 8 << 20


def palu_decode_attn_noalloc(cfg: PaluConfig, q, q_pos, zk_pool, zv_pool, zk_scales, zv_scales,
                             pos_pool, page_table, seq_lens, num_pages: int, B_k, B_v, out, lse,
                             num_splits: int = 0, stream=None, report_status: bool = False):
    """palu_decode_attn without a caller workspace (the library's fixed device array).

    report_status=True waits for the stream and raises on a device-detected fault.
    """
    batch = q.shape[0]
    max_pages = page_table.shape[1]
    detail = ctypes.c_int32()
    st = load().palu_decode_attn_noalloc(
        ctypes.byref(cfg), batch, _ptr(q), _ptr(q_pos), _ptr(zk_pool), _ptr(zv_pool),
        _ptr(zk_scales), _ptr(zv_scales), _ptr(pos_pool), _ptr(page_table), max_pages,
        _ptr(seq_lens), num_pages, _ptr(B_k), _ptr(B_v), _ptr(out), _ptr(lse), num_splits,
        _stream(stream), ctypes.byref(detail) if report_status else None)
    _check(st, "palu_decode_attn_noalloc")


# ---------------------------------------------------------------- planning, sparse steps, verification
# These calls check shapes and element types of every tensor, take the device from the tensors (it
# need not be the current one) and, without a stream, run on that device's current stream.
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


_get_device, _is_contiguous, _data_ptr = torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr


class _Args:
    """Checks the tensors of one call and gives their addresses.  The workspace names the device."""

    __slots__ = ("where", "device", "wrong")

    def __init__(self, where: str, workspace):
        if not isinstance(workspace, torch.Tensor):
            raise TypeError(f"{where}: workspace must be a torch.Tensor")
        self.where = where
        self.device = workspace.get_device()
        self.wrong = None            # what is not where the workspace is (told once shapes and types are known good)

    def __call__(self, name, t, dtype, shape=None):
        if t is None:
            return None
        if (isinstance(t, torch.Tensor) and t.get_device() == self.device >= 0 and t.is_contiguous() and
                (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape)):
            return t.data_ptr()
        return self._elsewhere(name, self._sound(name, t, dtype, shape))

    def take(self, names, tensors, dtypes, shapes):
        """Addresses of several tensors: what __call__ does for each, in a few passes over all of them
        (half the host time of a small call is spent on these checks)."""
        try:
            if (list(map(_get_device, tensors)) == [self.device] * len(tensors) and self.device >= 0 and
                    all(map(_is_contiguous, tensors)) and [t.dtype for t in tensors] == dtypes and
                    [t.shape for t in tensors] == shapes):
                return list(map(_data_ptr, tensors))
        except TypeError:
            pass
        return [self(*a) for a in zip(names, tensors, dtypes, shapes)]

    def _sound(self, name, t, dtype, shape):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: {name} must be a torch.Tensor or None")
        if dtype is not None and t.dtype is not dtype:
            raise ValueError(f"{self.where}: {name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{self.where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{self.where}: {name} must be contiguous")
        return t

    def _elsewhere(self, name, t):
        if t.numel() == 0:
            return None
        self.wrong = f"{name} must live in CUDA device memory" if not t.is_cuda else \
            f"{name} is on {t.device}, the workspace on device {self.device}"
        return None

    def rows(self, name, t, dtype, shape):
        """Address and row stride of [batch][rows][width] probabilities; rows may be padded."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.where}: {name} must be a torch.Tensor")
        if t.dtype is not dtype:
            raise ValueError(f"{self.where}: {name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{self.where}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        b, n, width = shape
        sb, ld, se = t.stride()
        ld = ld if n > 1 else sb if b > 1 else width          # a dimension of one has no stride to keep to
        if (width > 1 and se != 1) or (b > 1 and sb != n * ld) or ld < width:
            raise ValueError(f"{self.where}: rows of {name} must be contiguous and evenly spaced")
        if t.get_device() == self.device >= 0:
            return t.data_ptr(), ld
        return self._elsewhere(name, t), ld

    def call(self, fn, *args, stream=None):
        if self.device < 0:
            self.wrong = "workspace must live in CUDA device memory"
        if self.wrong is not None:
            raise ValueError(f"{self.where}: {self.wrong}")
        if self.device == torch.cuda.current_device():
            status = fn(*args, self._stream(stream))
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, self._stream(stream))
        if status != 0:
            raise PaluError(status, self.where)

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _size(where: str, *args) -> int:
    out = ctypes.c_size_t()
    _check(getattr(load(), where)(*args, ctypes.byref(out)), where)
    return int(out.value)


def palu_plan_workspace_size(batch: int) -> int:
    return _size("palu_plan_workspace_size", batch)


def palu_plan_append(page_size: int, num_new, seq_lens, page_table, free_pages, num_free, slot_mapping, positions,
                     row_starts, taken, workspace, stream=None):
    """Pages, slots and positions of the tokens every sequence appends (or drops: negative num_new).

    num_new, seq_lens [batch], page_table [batch][max_pages], free_pages [num_pages] (a stack of
    num_free[0] unused pages), slot_mapping and positions [n_rows]; seq_lens, page_table, free_pages
    and num_free are updated.  row_starts [batch + 1] and taken [batch] may be None.
    """
    A = _Args("palu_plan_append", workspace)
    batch, max_pages = page_table.shape
    one, rows = (batch,), (slot_mapping.numel(),)
    state = A.take(_PLAN, (num_new, seq_lens, page_table, free_pages, num_free, slot_mapping, positions), [_I32] * 7,
                   [one, one, (batch, max_pages), (free_pages.numel(),), (1,), rows, rows])
    A.call(load().palu_plan_append, page_size, batch, max_pages, free_pages.numel(), rows[0], *state,
           A("row_starts", row_starts, _I32, (batch + 1,)), A("taken", taken, _I32, one),
           A("workspace", workspace, None), workspace.numel() * workspace.element_size(), stream=stream)


_PLAN = ("num_new", "seq_lens", "page_table", "free_pages", "num_free", "slot_mapping", "positions")
_PROBS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def palu_verify_workspace_size(batch: int, num_drafts: int, vocab: int) -> int:
    return _size("palu_verify_workspace_size", batch, num_drafts, vocab)


def palu_verify_drafts(target_probs, draft_probs, draft_tokens, draft_lens, u_accept, u_sample, tokens, num_accepted,
                       rollback, workspace, stream=None):
    """Accept drafts against the target's probabilities and draw the token after them.

    target_probs [batch][D + 1][V], draft_probs [batch][D][V] or None (certain drafts), both float32,
    float16 or bfloat16 with evenly spaced rows (a slice of padded rows will do); draft_tokens and
    u_accept [batch][D], draft_lens [batch] or None, u_sample [batch]; tokens [batch][D + 1],
    num_accepted and rollback (or None) [batch] are written.
    """
    A = _Args("palu_verify_drafts", workspace)
    batch, n, vocab = target_probs.shape
    if target_probs.dtype not in _PROBS:
        raise ValueError(f"palu_verify_drafts: probabilities must be float32, float16 or bfloat16, "
                         f"got {target_probs.dtype}")
    one, D = (batch,), n - 1
    p, p_ld = A.rows("target_probs", target_probs, target_probs.dtype, (batch, n, vocab))
    q, q_ld = (None, 0) if draft_probs is None or D == 0 else \
        A.rows("draft_probs", draft_probs, target_probs.dtype, (batch, D, vocab))
    drafts, uniform, sample, out, accepted = A.take(
        _VERIFY, (draft_tokens, u_accept, u_sample, tokens, num_accepted), [_I32, _F32, _F32, _I32, _I32],
        [(batch, D), (batch, D), one, (batch, n), one])
    A.call(load().palu_verify_drafts, _PROBS[target_probs.dtype], batch, D, vocab, p, p_ld, q, q_ld,
           drafts, A("draft_lens", draft_lens, _I32, one), uniform, sample, out, accepted,
           A("rollback", rollback, _I32, one), A("workspace", workspace, None),
           workspace.nbytes, stream=stream)


_VERIFY = ("draft_tokens", "u_accept", "u_sample", "tokens", "num_accepted")
_ACT_TORCH = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}


class _Layer(NamedTuple):
    """What the checks of these calls take from a config and its ranks."""

    act: torch.dtype
    groups: int
    heads: int
    head_dim: int
    bounds: int          # entries of a page's bounds
    rows_k: int          # entries of B_k, B_v
    rows_v: int
    zk: int              # bytes per page of each pool
    zv: int
    zks: int
    zvs: int
    pos: int


def _page_bytes(cfg: PaluConfig, ranks) -> tuple[int, int]:
    """Bytes of one page of a latent pool and of its int4 scale pool, for the groups' ranks."""
    if cfg.latent_dtype != 3:
        return cfg.page_size * sum(ranks) * (4 if cfg.latent_dtype == 0 else 2), 0
    return cfg.page_size * sum(ranks) // 2, cfg.page_size * sum((r // 32 * 2 + 15) // 16 * 16 for r in ranks)


_uniform: dict[bytes, _Layer] = {}       # by the config's bytes: constants of a config, not of a call


def _layer(cfg: PaluConfig, ranks_k=None, ranks_v=None) -> _Layer:
    if (ranks_k is None) != (ranks_v is None):
        raise ValueError("ranks_k and ranks_v must be given together")
    if ranks_k is None:
        found = _uniform.get(bytes(cfg))
        if found is not None:
            return found
    G = cfg.num_heads // max(1, cfg.group_size)
    rk, rv = ((cfg.rank_k,) * G, (cfg.rank_v,) * G) if ranks_k is None else (ranks_k, ranks_v)
    if len(rk) != G or len(rv) != G:
        raise ValueError(f"ranks of {G} head groups expected, got {len(rk)} and {len(rv)}")
    (zk, zks), (zv, zvs) = _page_bytes(cfg, rk), _page_bytes(cfg, rv)
    width = cfg.group_size * cfg.head_dim
    made = _Layer(_ACT_TORCH.get(cfg.act_dtype), G, cfg.num_heads, cfg.head_dim, 2 * G * width, sum(rk) * width,
                  sum(rv) * width, zk, zv, zks, zvs, 4 * cfg.page_size)
    if ranks_k is None and len(_uniform) < 256:
        _uniform[bytes(cfg)] = made
    return made


def _pool(A, name, pool, num_pages, page_bytes, dtype=None):
    """A cache pool that holds at least num_pages pages (latents and scales: bytes of any type)."""
    if pool is None:
        return None
    if pool.nbytes < num_pages * page_bytes:
        raise ValueError(f"{A.where}: {name} holds fewer than {num_pages} pages")
    return A(name, pool, dtype)


def _sized(A, name, t, dtype, entries):
    """A tensor of exactly `entries` entries, whatever its shape."""
    if t.numel() != entries:
        raise ValueError(f"{A.where}: {name} must hold {entries} entries, got {t.numel()}")
    return A(name, t, dtype)


def _bounds(A, bounds, dtype, entries):
    if bounds.numel() < entries:
        raise ValueError(f"{A.where}: bounds holds fewer pages than the cache")
    return A("bounds", bounds, dtype)


def palu_page_bounds_bytes(cfg: PaluConfig) -> int:
    """Bytes of one page of the bounds pool [num_pages][G][2][group width], act dtype."""
    return _size("palu_page_bounds_bytes", ctypes.byref(cfg))


def palu_page_bounds_workspace_size(cfg: PaluConfig, batch: int, max_pages: int) -> int:
    return _size("palu_page_bounds_workspace_size", ctypes.byref(cfg), batch, max_pages)


def palu_page_bounds(cfg: PaluConfig, first, zk_pool, zk_scales, pos_pool, page_table, seq_lens, num_pages: int, B_k,
                     bounds, workspace, ranks_k=None, stream=None):
    """Rebuild the key bounds of the pages holding tokens first[b] .. seq_lens[b] - 1 (first None: all)."""
    A, L = _Args("palu_page_bounds", workspace), _layer(cfg, ranks_k, ranks_k)
    batch, max_pages = page_table.shape
    table, lens = A.take(("page_table", "seq_lens"), (page_table, seq_lens), [_I32, _I32], [(batch, max_pages), (batch,)])
    A.call(load().palu_page_bounds, ctypes.byref(cfg), _ranks(ranks_k), batch, A("first", first, _I32, (batch,)),
           _pool(A, "zk_pool", zk_pool, num_pages, L.zk), _pool(A, "zk_scales", zk_scales, num_pages, L.zks),
           _pool(A, "pos_pool", pos_pool, num_pages, L.pos, _I32), table, max_pages, lens, num_pages,
           _sized(A, "B_k", B_k, L.act, L.rows_k), _bounds(A, bounds, L.act, num_pages * L.bounds),
           A("workspace", workspace, None), workspace.nbytes, stream=stream)


def palu_select_workspace_size(cfg: PaluConfig, batch: int, num_queries: int, max_pages: int) -> int:
    return _size("palu_select_workspace_size", ctypes.byref(cfg), batch, num_queries, max_pages)


def palu_select_pages(cfg: PaluConfig, q, q_pos, bounds, pos_pool, page_table, seq_lens, num_pages: int,
                      num_first: int, num_last: int, page_list, page_counts, page_scores, workspace, stream=None):
    """The pages of largest score bound for every query and head group.

    q [batch][Q][H][d_h], q_pos [batch][Q]; page_list [batch][Q][G][list_len] (ascending, then -1),
    page_counts [batch][Q][G] and page_scores (like page_list, or None) are written.
    """
    A, L = _Args("palu_select_pages", workspace), _layer(cfg)
    batch, Q = q_pos.shape
    G, max_pages, keep = L.groups, page_table.shape[1], page_list.shape[-1]
    query, at, table, lens, lists, counts = A.take(
        _SELECT, (q, q_pos, page_table, seq_lens, page_list, page_counts), [L.act, _I32, _I32, _I32, _I32, _I32],
        [(batch, Q, L.heads, L.head_dim), (batch, Q), (batch, max_pages), (batch,), (batch, Q, G, keep), (batch, Q, G)])
    A.call(load().palu_select_pages, ctypes.byref(cfg), batch, Q, query, at,
           _bounds(A, bounds, L.act, num_pages * L.bounds), A("pos_pool", pos_pool, _I32), table, max_pages, lens,
           num_pages, num_first, num_last, keep, lists, counts,
           A("page_scores", page_scores, _F32, (batch, Q, G, keep)), A("workspace", workspace, None),
           workspace.nbytes, stream=stream)


_SELECT = ("q", "q_pos", "page_table", "seq_lens", "page_list", "page_counts")


def palu_decode_pages_workspace_size(cfg: PaluConfig, batch: int, num_queries: int, list_len: int,
                                     num_splits: int = 0, ranks_k=None, ranks_v=None) -> int:
    _layer(cfg, ranks_k, ranks_v)        # checks the number of ranks
    return _size("palu_decode_pages_workspace_size", ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v), batch,
                 num_queries, list_len, num_splits)


def palu_decode_attn_pages(cfg: PaluConfig, q, q_pos, zk_pool, zv_pool, zk_scales, zv_scales, pos_pool, page_table,
                           seq_lens, page_list, page_counts, num_pages: int, B_k, B_v, out, lse, workspace,
                           num_splits: int = 0, ranks_k=None, ranks_v=None, stream=None):
    """Decode step over listed pages: query j of sequence b attends, in group g, to the tokens of the
    logical pages page_list[b][j][g][:page_counts[b][j][g]] (strictly ascending).

    q and out [batch][Q][H][d_h], q_pos [batch][Q], lse [batch][Q][H] or None; Q > 1 is causal by position.
    """
    A, L = _Args("palu_decode_attn_pages", workspace), _layer(cfg, ranks_k, ranks_v)
    batch, Q = q_pos.shape
    G, max_pages, keep, rows = L.groups, page_table.shape[1], page_list.shape[-1], (batch, Q, L.heads, L.head_dim)
    query, at, table, lens, lists, counts, result = A.take(
        _ATTEND, (q, q_pos, page_table, seq_lens, page_list, page_counts, out),
        [L.act, _I32, _I32, _I32, _I32, _I32, L.act],
        [rows, (batch, Q), (batch, max_pages), (batch,), (batch, Q, G, keep), (batch, Q, G), rows])
    A.call(load().palu_decode_attn_pages, ctypes.byref(cfg), _ranks(ranks_k), _ranks(ranks_v), batch, Q, query, at,
           _pool(A, "zk_pool", zk_pool, num_pages, L.zk), _pool(A, "zv_pool", zv_pool, num_pages, L.zv),
           _pool(A, "zk_scales", zk_scales, num_pages, L.zks), _pool(A, "zv_scales", zv_scales, num_pages, L.zvs),
           _pool(A, "pos_pool", pos_pool, num_pages, L.pos, _I32), table, max_pages, lens, lists, counts, keep, num_pages,
           _sized(A, "B_k", B_k, L.act, L.rows_k), _sized(A, "B_v", B_v, L.act, L.rows_v), result,
           A("lse", lse, _F32, rows[:3]), A("workspace", workspace, None), workspace.nbytes, num_splits, stream=stream)


_ATTEND = ("q", "q_pos", "page_table", "seq_lens", "page_list", "page_counts", "out")


def palu_get_device_status(workspace, stream=None) -> tuple[int, int]:
    """(status, detail) of the device status word; clears it."""
    detail = ctypes.c_int32()
    st = load().palu_get_device_status(_ptr(workspace), _stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


@dataclass
class LatentCache:
    """Device buffers of a paged latent cache for one layer (caller-owned memory).

    Pools are uint8 tensors of num_pages pages each, laid out as include/palu.h
    states; ``view_*`` give typed views for inspection.
    """

    cfg: PaluConfig
    num_pages: int
    zk: torch.Tensor
    zv: torch.Tensor
    zks: torch.Tensor | None
    zvs: torch.Tensor | None
    pos: torch.Tensor | None
    ranks_k: tuple | None = None     # per-group ranks (None: the config's for every group)
    ranks_v: tuple | None = None

    @classmethod
    def allocate(cls, cfg: PaluConfig, num_pages: int, device="cuda", with_positions=False,
                 fill=None, ranks_k=None, ranks_v=None) -> "LatentCache":
        """Pools for num_pages pages; with ranks_k / ranks_v, the layout of a layer whose
        groups carry their own ranks (each page holds every group's block back to back)."""
        if ranks_k is None:
            kb, vb, ksb, vsb = palu_cache_strides(cfg)
        else:
            kb, vb, ksb, vsb, _, _ = palu_cache_strides_ranked(cfg, ranks_k, ranks_v)
        mk = (lambda n: torch.empty(n, dtype=torch.uint8, device=device)) if fill is None else \
            (lambda n: torch.full((n,), fill, dtype=torch.uint8, device=device))
        zks = mk(num_pages * ksb) if ksb else None
        zvs = mk(num_pages * vsb) if vsb else None
        pos = torch.zeros(num_pages * cfg.page_size, dtype=torch.int32, device=device) \
            if with_positions else None
        return cls(cfg, num_pages, mk(num_pages * kb), mk(num_pages * vb), zks, zvs, pos,
                   None if ranks_k is None else tuple(ranks_k), None if ranks_v is None else tuple(ranks_v))
