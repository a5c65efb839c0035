"""Plain 64-bit forms of the calls around a shared or forked prompt, and bounds on what
rounding may do to them, for the GPU tests (torch float64, one head or row at a time)."""
from __future__ import annotations

import math

import torch

from mixed_precision_kv_arkv_b200 import abi
from mixed_precision_kv_arkv_b200.cache import LayerCache, make_cfg

FP8 = {abi.ARKV_FMT_E4M3: torch.float8_e4m3fn, abi.ARKV_FMT_E5M2: torch.float8_e5m2}
FIELDS16 = ("k16", "v16", "pos16", "mu16", "m2_16")
FIELDS8 = ("k8", "v8", "sk", "sv", "pos8", "mu8", "m2_8")


def cfg(batch, hq, hkv, d, cap16=1, cap8=1, window=16, n_obs=16, fmt="e4m3", early=False):
    return make_cfg(batch, hq, hkv, d, window, n_obs, 1.0, 0.5, cap16, cap8, fmt, early)


def random_cache(c: abi.arkv_cfg, n16, n8, dev, seed, poison=True) -> LayerCache:
    """A cache with n16[s], n8[s] live slots in the rows of sequence s.  The slots past them hold
    NaN bit patterns (poison), which no call may let through."""
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = LayerCache(c, dev)
    d, dt = c.head_dim, FP8[c.quant_format]
    rn = lambda *s: torch.randn(s, generator=g, device=dev)
    if poison:
        for f in ("k16", "v16", "sk", "sv", "mu16", "m2_16", "mu8", "m2_8"):
            getattr(cache, f).fill_(float("nan"))
        cache.k8.fill_(0x7F), cache.v8.fill_(0xFF)
    fmax = 448.0 if c.quant_format == abi.ARKV_FMT_E4M3 else 57344.0
    for r in range(c.batch * c.hkv):
        a, b = n16[r // c.hkv], n8[r // c.hkv]
        cache.k16[r, :a], cache.v16[r, :a] = rn(a, d).bfloat16(), rn(a, d).bfloat16()
        for x in "kv":
            val = rn(b, d) * torch.exp(rn(b, 1))
            s = val.abs().amax(-1) / fmax
            getattr(cache, x + "8")[r, :b] = (val / s[:, None]).to(dt).view(torch.uint8)
            getattr(cache, "s" + x)[r, :b] = s
        for key, n in (("16", a), ("8", b)):
            getattr(cache, "pos" + key)[r, :n] = torch.randperm(n, generator=g, device=dev).int()
            getattr(cache, "mu" + key)[r, :n] = torch.rand(n, generator=g, device=dev).double()
            getattr(cache, "m2_" + key)[r, :n] = torch.rand(n, generator=g, device=dev).double()
        cache.n_bf16[r], cache.n_fp8[r] = a, b
    return cache


def row_tokens(cache: LayerCache, r):
    """K^ and V^ of a row's live tokens, float64 (counts clamped to the capacities)."""
    c = cache.cfg
    dt = FP8[c.quant_format]
    a, b = min(int(cache.n_bf16[r]), c.cap_bf16), min(int(cache.n_fp8[r]), c.cap_fp8)
    one = lambda x: torch.cat([getattr(cache, x + "16")[r, :a].double(),
                               getattr(cache, x + "8")[r, :b].view(dt).double()
                               * getattr(cache, "s" + x)[r, :b].double()[:, None]])
    return one("k"), one("v")


def prefix_attn(c: abi.arkv_cfg, prefix: LayerCache, q, starts, o_own=None, ml_own=None):
    """(o, ml, o_bound, m_bound, l_rel_bound) of arkv_prefix_attn in float64.

    The bounds count roundings.  u = 2^-8 is bf16's half step, relative.
      logits: float32 accumulation over D products, each partial sum at most S = sum |q_i k_i|:
        D 2^-24 S in the worst order, and scale and log2 factors on top: (D + 8) 2^-24 S
      M: that logit bound of the largest one
      p = exp((raw - M) / sqrt(D)): twice the logit bound / sqrt(D), the exponential's own 2^-20, and
        2^-21 |raw - M| / sqrt(D) for the scaled argument's rounding, weighted by p: at most 2^-21 (x e^-x <= 1)
      o: P rounded once (u), the sums over n tokens in float32 (n 2^-24, at most 2^-10), o rounded (u)"""
    d, G, hkv = c.head_dim, c.hq // c.hkv, c.hkv
    n = c.batch
    f64 = dict(dtype=torch.float64, device=q.device)
    o, ml = torch.zeros((n, c.hq, d), **f64), torch.zeros((n * hkv, 4, 2), **f64)
    ob, mb, lb = torch.zeros_like(o), torch.zeros((n * hkv, 4), **f64), torch.zeros((n * hkv, 4), **f64)
    ml[..., 0] = float("-inf")
    pre_of = [-1] * n
    for p in range(len(starts) - 1):
        for b in range(max(0, starts[p]), min(n, starts[p + 1])):
            pre_of[b] = p
    u = 2.0 ** -8
    for b in range(n):
        for g in range(hkv):
            if pre_of[b] >= 0:
                K, V = row_tokens(prefix, pre_of[b] * hkv + g)
            else:
                K = V = torch.zeros((0, d), **f64)
            hs = slice(g * G, (g + 1) * G)
            Q = q[b, hs].double()
            raw = Q @ K.T
            S = Q.abs() @ K.abs().T
            M = raw.amax(-1) if raw.shape[1] else torch.full((G,), float("-inf"), **f64)
            Lo = torch.zeros(G, **f64)
            Oo = torch.zeros((G, d), **f64)
            Mo = torch.full((G,), float("-inf"), **f64)
            if o_own is not None:
                Lo, Oo = ml_own[b * hkv + g, :G, 1].double(), o_own[b, hs].double()
                Mo = torch.where(Lo != 0, ml_own[b * hkv + g, :G, 0].double(), Mo)
                M = torch.maximum(M, Mo)
            fin = torch.where(torch.isinf(M), torch.zeros_like(M), M)
            P = torch.exp((raw - fin[:, None]) / math.sqrt(d))
            W = torch.where(Lo != 0, Lo * torch.exp((Mo - fin) / math.sqrt(d)), torch.zeros_like(Lo))
            L = P.sum(-1) + W
            Z = torch.where(L == 0, torch.ones_like(L), L)[:, None]
            out = (P @ V + W[:, None] * torch.where((W == 0)[:, None], torch.zeros_like(Oo), Oo)) / Z
            mass = (P @ V.abs() + (W[:, None] * Oo.abs() if o_own is not None else 0.0)) / Z
            top = S.amax(-1) if S.shape[1] else torch.zeros(G, **f64)
            e_raw = (d + 8) * 2.0 ** -24 * top
            e_p = 2 * e_raw / math.sqrt(d) + 2.0 ** -20 + 2.0 ** -21
            e_sum = min(K.shape[0] * 2.0 ** -24, 2.0 ** -10)
            o[b, hs] = out
            ob[b, hs] = u * out.abs() * (1 + 2 * u) + (u + 2 * e_p + 2 * e_sum)[:, None] * mass
            ml[b * hkv + g, :G] = torch.stack([M, L], -1)
            mb[b * hkv + g, :G] = e_raw
            lb[b * hkv + g, :G] = e_p + e_sum
    return o, ml, ob, mb, lb


def check_prefix(c, got_o, got_ml, ref, rows=None):
    o, ml, ob, mb, lb = ref
    G = c.hq // c.hkv
    err = (got_o.double() - o).abs()
    assert torch.isfinite(got_o).all()
    bad = err > ob + 1e-30
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((err / (ob + 1e-30)).max()))
    if got_ml is None:
        return
    gm, gl = got_ml[:, :G, 0].double(), got_ml[:, :G, 1].double()
    rm, rl, mb, lb = ml[:, :G, 0], ml[:, :G, 1], mb[:, :G], lb[:, :G]
    none = rl == 0
    assert (gl[none] == 0).all() and (gm[none] == float("-inf")).all()
    assert ((gm - rm).abs()[~none] <= mb[~none] + 2.0 ** -23 * rm.abs()[~none]).all()
    # L goes with the M it is relative to: compare M / sqrt(D) + ln L
    sc = 1.0 / math.sqrt(c.head_dim)
    lse, ref_lse = gm * sc + gl.log(), rm * sc + rl.log()
    tol = lb + mb * sc + 2.0 ** -22 * (1.0 + rm.abs() * sc)
    assert ((lse - ref_lse).abs()[~none] <= tol[~none]).all()


def qk_norm_rope(c, n_tok, qkv, pos0, step, lengths, wq, wk, eps, freq, rot, interleaved):
    """(q, k, v, bound_q, bound_k) in float64 for the live tokens, [batch, heads, n_tok, D]; zero elsewhere.
    Bound of an output y = a cos f - b sin f: bf16's half step 2^-8 |y|; the norm, weight and products in float32,
    the angle (turns to 2^-32, its float32 value, sine and cosine) together at most 2^-20 (|a| + |b|)."""
    b, hq, hkv, d = c.batch, c.hq, c.hkv, c.head_dim
    x = qkv[:, :(hq + 2 * hkv) * d].double().reshape(b, n_tok, hq + 2 * hkv, d)
    out = []
    t = torch.arange(n_tok, device=qkv.device, dtype=torch.float64)
    pos = (pos0.double() if pos0 is not None else torch.zeros(b, device=qkv.device, dtype=torch.float64))[:, None] + step + t
    live = (torch.arange(n_tok, device=qkv.device) < lengths[:, None])[:, None, :, None]
    for lo, hi, w in ((0, hq, wq), (hq, hq + hkv, wk), (hq + hkv, hq + 2 * hkv, None)):
        y = x[:, :, lo:hi].clone()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
        mag = y.abs()
        if lo < hq + hkv and rot:
            f = (pos[..., None] * freq)[:, :, None, :]
            i = torch.arange(rot // 2, device=qkv.device)
            ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            a, bb = y[..., ia].clone(), y[..., ib].clone()
            y[..., ia], y[..., ib] = a * f.cos() - bb * f.sin(), a * f.sin() + bb * f.cos()
            mag[..., ia] = mag[..., ib] = a.abs() + bb.abs()
        y, mag = y.transpose(1, 2), mag.transpose(1, 2)
        out.append((torch.where(live, y, 0.0), torch.where(live, 2.0 ** -8 * y.abs() + 2.0 ** -20 * mag, 0.0)))
    (q, bq), (k, bk), (v, _) = out
    return q, k, v, bq, bk
