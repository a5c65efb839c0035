"""Device-memory plumbing around libarkv: torch tensors for one layer's packed
cache and workspaces, and per-layer drivers that issue the C-ABI calls of the
decode path in order: a sequence's own step, a step of branches that share a
prefix, forks of a cache, and the projection's norm and rotation before them.
Nothing here computes any part of the method.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import abi


def make_cfg(batch, hq, hkv, head_dim, window, n_obs, gamma, budget_frac, cap_bf16, cap_fp8,
             quant_format="e4m3", early_start=False):
    return abi.arkv_cfg(batch, hq, hkv, head_dim, window, n_obs, float(gamma), float(budget_frac),
                        cap_bf16, cap_fp8, abi.FORMATS[quant_format], int(bool(early_start)))


class LayerCache:
    """The tri-state cache of one layer (see include/arkv.h, Layout)."""

    def __init__(self, cfg: abi.arkv_cfg, device):
        R, D = cfg.batch * cfg.hkv, cfg.head_dim
        co, cq = cfg.cap_bf16, cfg.cap_fp8
        i32, f32, f64, u8 = torch.int32, torch.float32, torch.float64, torch.uint8
        self.cfg = cfg
        self.k16 = torch.zeros((R, co, D), dtype=torch.bfloat16, device=device)
        self.v16 = torch.zeros((R, co, D), dtype=torch.bfloat16, device=device)
        self.pos16 = torch.zeros((R, co), dtype=i32, device=device)
        self.mu16 = torch.zeros((R, co), dtype=f64, device=device)
        self.m2_16 = torch.zeros((R, co), dtype=f64, device=device)
        self.k8 = torch.zeros((R, cq, D), dtype=u8, device=device)
        self.v8 = torch.zeros((R, cq, D), dtype=u8, device=device)
        self.sk = torch.zeros((R, cq), dtype=f32, device=device)
        self.sv = torch.zeros((R, cq), dtype=f32, device=device)
        self.pos8 = torch.zeros((R, cq), dtype=i32, device=device)
        self.mu8 = torch.zeros((R, cq), dtype=f64, device=device)
        self.m2_8 = torch.zeros((R, cq), dtype=f64, device=device)
        self.n_bf16 = torch.zeros((R,), dtype=i32, device=device)
        self.n_fp8 = torch.zeros((R,), dtype=i32, device=device)
        self.status = torch.zeros((1,), dtype=i32, device=device)
        self.c = abi.arkv_layer_cache(*[getattr(self, n).data_ptr() for n, _ in
                                        abi.arkv_layer_cache._fields_])

    def nbytes(self) -> int:
        return sum(getattr(self, n).numel() * getattr(self, n).element_size()
                   for n, _ in abi.arkv_layer_cache._fields_)


class Workspace:
    """A zero-filled, 256-byte aligned device workspace of a given size."""

    def __init__(self, nbytes: int, device):
        self.buf = torch.zeros(max(int(nbytes), 1) + 256, dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        self.off = (-base) % 256
        self.ptr = base + self.off
        self.nbytes = int(nbytes)


def stream_ptr(stream=None) -> int:
    """The raw handle of `stream`, or of the current device's current stream (without the stream
    object that torch.cuda.current_stream() makes: 0.2 us instead of 3.3)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


@dataclass
class LayerState:
    """What the decode loop of one layer holds on the device."""
    cfg: abi.arkv_cfg
    cache: LayerCache
    ws_decode: Workspace
    ws_reassign: Workspace
    r: float


def new_layer_state(cfg: abi.arkv_cfg, r: float, device) -> LayerState:
    return LayerState(cfg, LayerCache(cfg, device),
                      Workspace(abi.arkv_workspace_bytes(cfg, abi.ARKV_WS_DECODE), device),
                      Workspace(abi.arkv_workspace_bytes(cfg, abi.ARKV_WS_REASSIGN), device), float(r))


def decode_step(st: LayerState, step: int, q, k_new, v_new, ctx_len, o, reassign_interval: int,
                stream=None, tier_dbg=None):
    """One decode step of one layer: append + attend, score update, and a
    reassignment when (step + 1) % reassign_interval == 0."""
    s = stream_ptr(stream)
    abi.arkv_decode_attn(st.cfg, step, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                         ctx_len.data_ptr(), st.cache.c, o.data_ptr(), st.ws_decode.ptr,
                         st.ws_decode.nbytes, s)
    abi.arkv_score_update(st.cfg, step, ctx_len.data_ptr(), st.cache.c, st.ws_decode.ptr,
                          st.ws_decode.nbytes, s)
    if (step + 1) % reassign_interval == 0:
        abi.arkv_reassign(st.cfg, step, st.r, ctx_len.data_ptr(), st.cache.c,
                          tier_dbg.data_ptr() if tier_dbg is not None else None,
                          st.ws_reassign.ptr, st.ws_reassign.nbytes, s)


def _on_device(t: torch.Tensor, stream):
    """The device guard and raw stream of a call on t's device."""
    if t.device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {t.device}")
    s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(t.device.index)
    return torch.cuda.device(t.device), s


def _ptr(t):
    return None if t is None else t.data_ptr()


def _expect(name, t, dtype, device, numel):
    """A tensor that a call reads or writes by its address alone."""
    if t.dtype != dtype or t.device != device or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} on {device} with {numel} elements, not {t.dtype} on "
                         f"{t.device} of shape {tuple(t.shape)} and strides {t.stride()}")


def rope_frequencies(rot: int, theta: float, device) -> torch.Tensor:
    """theta ** (-2 i / rot) for the rot / 2 rotated pairs, float64 radians per position."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (float(theta) ** (-2.0 * i / max(rot, 1))).to(device)


def qk_norm_rope(cfg: abi.arkv_cfg, qkv, n_tok: int, freq, k, v, q=None, q_obs=None, *, q_weight=None,
                 k_weight=None, eps: float = 1e-6, interleaved=False, pos0=None, step: int = 0, length=None,
                 stream=None):
    """arkv_qk_norm_rope on torch tensors: qkv [batch * n_tok, >= (hq + 2 hkv) D] bf16 (unit stride in
    its last dimension), freq [rot / 2] float64 or None, k, v (and q) [batch, heads, n, D] bf16, q_obs [batch, hq,
    n_obs, D]; q_weight, k_weight [D] bf16, pos0, length [batch] int32.  All but qkv are contiguous."""
    b, hq, hkv, d = cfg.batch, cfg.hq, cfg.hkv, cfg.head_dim
    dev, bf16, width = qkv.device, torch.bfloat16, (hq + 2 * hkv) * d
    if qkv.dim() != 2 or qkv.stride(1) != 1 or qkv.shape[0] != b * n_tok or qkv.shape[1] < width or qkv.dtype != bf16:
        raise ValueError(f"qkv must be {bf16} [batch * n_tok, {width} or more] with unit stride in its last dimension")
    n = k.shape[2] if k.dim() == 4 else 0
    for name, t, shape in (("k", k, (b, hkv, n, d)), ("v", v, (b, hkv, n, d)), ("q", q, (b, hq, n, d)),
                           ("q_obs", q_obs, (b, hq, cfg.n_obs, d))):
        if t is not None and (t.shape != shape or t.dtype != bf16 or t.device != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous {bf16} of shape {shape} on {dev}")
    for name, t, dt, count in (("q_weight", q_weight, bf16, d), ("k_weight", k_weight, bf16, d),
                               ("pos0", pos0, torch.int32, b), ("length", length, torch.int32, b)):
        if t is not None:
            _expect(name, t, dt, dev, count)
    rot = 0
    if freq is not None:   # (rot <= head_dim is the library's check)
        rot = 2 * freq.numel()
        _expect("freq", freq, torch.float64, dev, rot // 2)
    guard, s = _on_device(qkv, stream)
    with guard:
        abi.arkv_qk_norm_rope(cfg, n_tok, qkv.data_ptr(), qkv.stride(0) if qkv.shape[0] > 1 else width, _ptr(pos0), step,
                              _ptr(length), _ptr(q_weight), _ptr(k_weight), eps, _ptr(freq), rot, int(bool(interleaved)), n,
                              _ptr(q), k.data_ptr(), v.data_ptr(), _ptr(q_obs), s)


def fork(dst: LayerCache, src: LayerCache, src_seq, stream=None):
    """arkv_cache_fork: sequence b of dst becomes a copy of sequence src_seq[b] of src (int32 tensor;
    abi.ARKV_SEQ_FREE, abi.ARKV_SEQ_KEEP).  dst may be src itself (see include/arkv.h)."""
    if src_seq.dtype != torch.int32 or src_seq.numel() != dst.cfg.batch or not src_seq.is_contiguous():
        raise ValueError("src_seq must be a contiguous int32 tensor with one entry per sequence of dst")
    if not (src_seq.device == dst.k16.device == src.k16.device):
        raise ValueError("src_seq and the two caches must be on one device")
    guard, s = _on_device(dst.k16, stream)
    with guard:
        abi.arkv_cache_fork(dst.cfg, dst.c, src.cfg, src.c, src_seq.data_ptr(), s)


@dataclass
class SharedPrefix:
    """A packed cache whose sequences are prefixes, shared by the branches of another layer state."""
    cache: LayerCache
    branch_start: torch.Tensor | None    # [prefixes + 1] int32, or None: one prefix, every branch
    ws: Workspace


def new_shared_prefix(branches: abi.arkv_cfg, cache: LayerCache, branch_start=None) -> SharedPrefix:
    """The prefixes in `cache` for the branches described by `branches`.  branch_start: a list or a tensor
    (a tensor on the device is taken as it is, its order is the caller's to keep)."""
    dev = cache.k16.device
    if branch_start is None:
        if cache.cfg.batch != 1:
            raise ValueError("branch_start must be given for several prefixes")
    else:
        starts = torch.as_tensor(branch_start)
        if starts.numel() != cache.cfg.batch + 1:
            raise ValueError("branch_start must have one entry per prefix and one more")
        if starts.device.type == "cpu" and (starts.diff() < 0).any():
            raise ValueError("branch_start must not decrease")
        branch_start = starts.to(dtype=torch.int32, device=dev).contiguous()
    nbytes = abi.arkv_prefix_workspace_bytes(branches, cache.cfg)
    if nbytes == 0:
        raise ValueError("the branches and the prefixes do not fit together: "
                         + abi.lib().arkv_last_error_string().decode())
    return SharedPrefix(cache, branch_start, Workspace(nbytes, dev))


def branch_step(st: LayerState, prefix: SharedPrefix, step: int, q, k_new, v_new, ctx_len, o_own, o,
                reassign_interval: int, stream=None, tier_dbg=None):
    """One decode step of one layer whose sequences share prefixes: append + attend to the own
    tokens (o_own, float32), attend to the prefix and join (o, bf16, and the heads' (max, sum) in
    the decode workspace), score update of the own tokens, and their reassignment when
    (step + 1) % reassign_interval == 0 (the prefix's bytes are part of the budget, see arkv_branch_reassign, which
    also says how to size the own cache).  ctx_len counts the prefix's tokens.  All tensors are contiguous:
    q, o_own, o [batch, hq, D], k_new, v_new [batch, hkv, D] (or any shape of as many elements)."""
    c, dev = st.cfg, st.cache.k16.device
    nq, nkv = c.batch * c.hq * c.head_dim, c.batch * c.hkv * c.head_dim
    for name, t, dt, n in (("q", q, torch.bfloat16, nq), ("k_new", k_new, torch.bfloat16, nkv),
                           ("v_new", v_new, torch.bfloat16, nkv), ("ctx_len", ctx_len, torch.int32, c.batch),
                           ("o_own", o_own, torch.float32, nq), ("o", o, torch.bfloat16, nq)):
        _expect(name, t, dt, dev, n)
    if tier_dbg is not None:
        _expect("tier_dbg", tier_dbg, torch.uint8, dev, c.batch * c.hkv * (c.cap_bf16 + c.cap_fp8))
    # what the later calls would refuse is refused before the first one appends
    need = abi.arkv_prefix_workspace_bytes(c, prefix.cache.cfg)
    if prefix.cache.k16.device != dev or need == 0 or prefix.ws.nbytes < need:
        raise ValueError("prefix must be on the device of the branches' cache and made for their configuration")
    if o.data_ptr() % 16:
        raise ValueError("o must be 16-byte aligned")
    guard, s = _on_device(q, stream)
    with guard:
        abi.arkv_decode_attn(st.cfg, step, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), ctx_len.data_ptr(),
                             st.cache.c, o_own.data_ptr(), st.ws_decode.ptr, st.ws_decode.nbytes, s)
        ml = abi.arkv_decode_ml(st.cfg, st.ws_decode.ptr, st.ws_decode.nbytes)
        abi.arkv_prefix_attn(st.cfg, prefix.cache.cfg, q.data_ptr(), prefix.cache.c, _ptr(prefix.branch_start),
                             o_own.data_ptr(), ml, o.data_ptr(), ml, prefix.ws.ptr, prefix.ws.nbytes, s)
        abi.arkv_score_update(st.cfg, step, ctx_len.data_ptr(), st.cache.c, st.ws_decode.ptr,
                              st.ws_decode.nbytes, s)
        if (step + 1) % reassign_interval == 0:
            abi.arkv_branch_reassign(st.cfg, step, st.r, ctx_len.data_ptr(), st.cache.c, prefix.cache.cfg, prefix.cache.c,
                                     _ptr(prefix.branch_start), _ptr(tier_dbg), st.ws_reassign.ptr,
                                     st.ws_reassign.nbytes, s)
