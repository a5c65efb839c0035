"""How exactly arkv_prefix_attn weighs the prefix's values: its probabilities carry 16 bits, as
arkv_decode_attn's do, whatever the number of tokens, prefixes and spare slots of the call.  A few
tokens of every row take nearly the whole softmax, so that one rounding of their probabilities to
bf16 would show beside the rounding of o itself.  And what such a call is made of: segments of many
tiles, a softmax reference that moves in a later tile, one and two tiles of query rows."""
from __future__ import annotations

import math

import pytest
import torch

from mixed_precision_kv_arkv_b200 import abi
from mixed_precision_kv_arkv_b200.build import build
from mixed_precision_kv_arkv_b200 import cache as C
from tests import plain_ops as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    abi.lib()


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def exact(c, prefix, q, starts):
    """(o, mass, M, L, S) of the prefix alone in float64: mass = sum p |v|, S = the largest sum |q_i k_i|."""
    n, hkv, G, d = c.batch, c.hkv, c.hq // c.hkv, c.head_dim
    f64 = dict(dtype=torch.float64, device=q.device)
    o, mass = torch.zeros((n, c.hq, d), **f64), torch.zeros((n, c.hq, d), **f64)
    M, L, S = (torch.zeros((n, c.hq), **f64) for _ in range(3))
    for p in range(len(starts) - 1):
        br = slice(starts[p], starts[p + 1])
        for g in range(hkv if starts[p + 1] > starts[p] else 0):
            K, V = R.row_tokens(prefix, p * hkv + g)
            hs = slice(g * G, (g + 1) * G)
            Q = q[br, hs].double()
            raw = Q @ K.T
            M[br, hs] = raw.amax(-1)
            w = torch.exp((raw - M[br, hs, None]) / math.sqrt(d))
            L[br, hs] = w.sum(-1)
            o[br, hs] = w @ V / L[br, hs, None]
            mass[br, hs] = w @ V.abs() / L[br, hs, None]
            S[br, hs] = (Q.abs() @ K.abs().T).amax(-1)
    return o, mass, M, L, S


def bounds(c, ref, tiles):
    """What rounding may do to o (by element) and to M / sqrt(D) + ln L (by head).
      accumulations of the tensor cores: 16 products at a time, at most 2^-22 of what they add up (float32's
        2^-24 for the sum and for the largest terms cut to its last place)
      logits: D / 16 accumulations of at most S, of the token and of the reference; a scale's 2^-24
      exponential and its argument: 2^-20 + 2^-21
      P: two bf16 parts; the first leaves at most 2^-8 p, the second rounds that once more: 2^-16
      sums: `tiles` of 64 tokens are a chain of 8 accumulations each (four of either part); the join adds
        the segments of a unit one by one in four quarters, at most 148 / 4 and 4
      o: one rounding to bf16, 2^-8, of the value as computed"""
    o, mass, M, L, S = ref
    d = c.head_dim
    e_raw = (d / 16 * 2.0 ** -22 + 2.0 ** -24) * S / math.sqrt(d)
    e_p = 2 * e_raw + 2.0 ** -20 + 2.0 ** -21
    e_sum = (8 * tiles + 41) * 2.0 ** -22
    pre = (2.0 ** -16 + 2 * e_p + 2 * e_sum)[..., None] * mass
    return 2.0 ** -8 * (o.abs() + pre) + pre, e_raw + e_p + e_sum + 2.0 ** -22 * (1 + M.abs() / math.sqrt(d))


def heavy_prefix(pc, n16, n8, dev, seed, heavy=4, level=12.0):
    """Caches whose rows have `heavy` tokens each (dealt over both segments) that queries along u weigh
    e^level times as much as the others, and u [hkv, D].  Their values alternate in sign, so that o is a
    difference of nearly equal terms, each with its probability's rounding."""
    prefix = R.random_cache(pc, n16, n8, dev, seed)
    g = gen(dev, seed + 1)
    hkv, d = pc.hkv, pc.head_dim
    u = torch.randn((hkv, d), generator=g, device=dev)
    u *= math.sqrt(d) / u.norm(dim=1, keepdim=True)
    fmax = 448.0 if pc.quant_format == abi.ARKV_FMT_E4M3 else 57344.0
    pick = torch.Generator().manual_seed(seed + 2)
    for r in range(pc.batch * hkv):
        a, b = n16[r // hkv], n8[r // hkv]
        w = torch.randn(d, generator=g, device=dev)
        for i, t in enumerate(torch.randperm(a + b, generator=pick)[:heavy].tolist()):
            k = (level + 0.2 * torch.rand((), generator=g, device=dev)) / math.sqrt(d) * u[r % hkv]
            v = w if i % 2 else -w
            if t < a:
                prefix.k16[r, t], prefix.v16[r, t] = k.bfloat16(), v.bfloat16()
                continue
            for name, x in (("k", k), ("v", v)):
                s = x.abs().max() / fmax
                getattr(prefix, name + "8")[r, t - a] = (x / s).to(R.FP8[pc.quant_format]).view(torch.uint8)
                getattr(prefix, "s" + name)[r, t - a] = s
    return prefix, u


def queries(c, u, dev, seed, noise=0.3):
    G = c.hq // c.hkv
    return (u.repeat_interleave(G, 0)[None] + noise * torch.randn((c.batch, c.hq, c.head_dim), generator=gen(dev, seed),
                                                                  device=dev)).bfloat16()


def run(c, prefix, q, starts=None):
    sp = C.new_shared_prefix(c, prefix, starts)
    o = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=q.device)
    ml = torch.full((c.batch * c.hkv, 4, 2), 5.0, device=q.device)
    abi.arkv_prefix_attn(c, prefix.cfg, q.data_ptr(), prefix.c, C._ptr(sp.branch_start), None, None, o.data_ptr(),
                         ml.data_ptr(), sp.ws.ptr, sp.ws.nbytes, C.stream_ptr())
    torch.cuda.synchronize()
    return o, ml


def check(c, got, ref, tiles):
    o, ml = got
    G = c.hq // c.hkv
    tol, tol_l = bounds(c, ref, tiles)
    err = (o.double() - ref[0]).abs()
    assert (err <= tol).all(), (int((err > tol).sum()), float((err / (tol + 1e-300)).max()))
    m, l = ml.view(c.batch, c.hkv, 4, 2)[:, :, :G].reshape(c.batch, c.hq, 2).double().unbind(-1)
    sc = 1 / math.sqrt(c.head_dim)
    lse, want = m * sc + l.log(), ref[2] * sc + ref[3].log()
    assert ((lse - want).abs() <= tol_l).all()


CASES = [
    # hq, hkv, D, fmt, n16, n8, spare slots, starts, branches, tiles in a CTA's run (at most)
    (8, 2, 64, "e4m3", [356], [292], 0, None, 2, 1),
    (8, 2, 64, "e4m3", [356], [292], 200000, None, 2, 1),          # the same tokens in a large allocation
    (32, 8, 128, "e4m3", [5921], [4739], 0, None, 4, 16),          # few rows of one tile
    (32, 8, 128, "e5m2", [5921], [4739], 0, None, 32, 16),         # a whole tile of rows
    (32, 8, 64, "e4m3", [9000], [9001], 0, None, 31, 24),
    (32, 8, 64, "e5m2", [9000], [9001], 0, None, 64, 24),          # two whole tiles of rows
    (32, 8, 128, "e4m3", [9000], [9001], 0, None, 63, 24),
    (12, 4, 128, "e5m2", [3000, 20, 900], [100, 4000, 2500], 40, [0, 3, 20, 42], 42, 16),
    (16, 8, 64, "e4m3", [356] * 8, [292] * 8, 3, [3 * i for i in range(9)], 24, 8),
]


@pytest.mark.parametrize("hq,hkv,d,fmt,n16,n8,spare,starts,branches,tiles", CASES)
def test_probabilities_keep_16_bits(cuda, hq, hkv, d, fmt, n16, n8, spare, starts, branches, tiles):
    pc = R.cfg(len(n16), hq, hkv, d, max(n16) + spare, max(n8) + spare, fmt=fmt)
    prefix, u = heavy_prefix(pc, n16, n8, cuda, 70)
    c = R.cfg(branches, hq, hkv, d)
    q = queries(c, u, cuda, 75)
    ref = exact(c, prefix, q, starts or [0, branches])
    check(c, run(c, prefix, q, starts), ref, tiles)
    assert int(prefix.status) == 0


def test_spare_slots_change_nothing(cuda):
    """The same tokens in a larger allocation: the same bits."""
    got = []
    for spare in (0, 100000):
        prefix, u = heavy_prefix(R.cfg(1, 8, 2, 128, 700 + spare, 900 + spare), [700], [900], cuda, 80)
        c = R.cfg(5, 8, 2, 128)
        got.append(run(c, prefix, queries(c, u, cuda, 81)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


RISING = [
    # D, queries a key head, prefixes, branches of each
    (128, 4, 32, 1),      # one tile of rows, few of them live
    (64, 1, 20, 6),       # one tile, more
    (128, 4, 20, 50),     # two tiles
    (64, 3, 20, 60),      # two tiles of 42 branches
]


def rising_prefix(pc, dev, seed, low=-104.0, high=104.0):
    """Rows whose logits (for queries along u, natural units) rise from low to high along the bf16 tokens and
    then the FP8 tokens; odd prefixes fall instead."""
    n16, n8 = pc.cap_bf16, pc.cap_fp8
    prefix, u = heavy_prefix(pc, [n16] * pc.batch, [n8] * pc.batch, dev, seed, heavy=0)
    g, d, hkv = gen(dev, seed + 3), pc.head_dim, pc.hkv
    fmax = 448.0 if pc.quant_format == abi.ARKV_FMT_E4M3 else 57344.0
    ramp = torch.linspace(low, high, n16 + n8, device=dev)[:, None] / math.sqrt(d)
    for r in range(pc.batch * hkv):
        k = ramp * u[r % hkv] * (1.0 if (r // hkv) % 2 == 0 else -1.0)
        k = k + 0.2 * torch.randn(k.shape, generator=g, device=dev)
        prefix.k16[r] = k[:n16].bfloat16()
        s = k[n16:].abs().amax(-1) / fmax
        prefix.k8[r], prefix.sk[r] = (k[n16:] / s[:, None]).to(R.FP8[pc.quant_format]).view(torch.uint8), s
    return prefix, u


@pytest.mark.parametrize("d,G,prefixes,branches", RISING)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_long_runs_with_a_rising_reference(cuda, d, G, prefixes, branches, fmt):
    """Units of 17 tiles (150 at least of them on 148 SMs), along which the logits rise by 300 log2 units: in
    every run the reference moves again and again (at a rise past 2^32 of it) and o is rescaled,
    between bf16 tiles, between FP8 tiles and from one kind to the other; in the odd prefixes the first tiles
    alone count.  Runs cross units and use every place of the ring and of the scales."""
    hkv = 8
    pc = R.cfg(prefixes, hkv * G, hkv, d, 515, 509, fmt=fmt)
    prefix, u = rising_prefix(pc, cuda, 85)
    c = R.cfg(prefixes * branches, hkv * G, hkv, d)
    starts = [branches * i for i in range(prefixes + 1)]
    q = queries(c, u, cuda, 95, noise=0.1)
    ref = exact(c, prefix, q, starts)
    first = run(c, prefix, q, starts)
    check(c, first, ref, 17)
    again = run(c, prefix, q, starts)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert int(prefix.status) == 0


@pytest.mark.parametrize("d,branches,prefixes", [(128, 4, 1), (64, 40, 1), (128, 1, 20), (64, 40, 20)])
def test_tokens_without_weight_first(cuda, d, branches, prefixes):
    """The first 130 tokens have logits of -inf, the others all of about -140 (e^-140 is past float32's
    range): the others make up the softmax.  A prefix of -inf alone has no weight: o = 0, (-inf, 0)."""
    hkv, G, n16, n8 = 8, 4, 400, 300
    pc = R.cfg(prefixes + 1, hkv * G, hkv, d, n16, n8)
    prefix, u = heavy_prefix(pc, [n16] * prefixes + [70], [n8] * prefixes + [0], cuda, 90, heavy=0)
    prefix.k16[prefixes * hkv:, :70, 0] = float("-inf")
    g = gen(cuda, 91)
    for r in range(prefixes * hkv):
        k = -140 / math.sqrt(d) * u[r % hkv] + 0.2 * torch.randn((n16 + n8, d), generator=g, device=cuda)
        prefix.k16[r] = k[:n16].bfloat16()
        prefix.k16[r, :130, 0] = float("-inf")
        s = k[n16:].abs().amax(-1) / 448.0
        prefix.k8[r], prefix.sk[r] = (k[n16:] / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), s
    c = R.cfg(prefixes * branches + 1, hkv * G, hkv, d)
    starts = [branches * i for i in range(prefixes + 1)] + [prefixes * branches + 1]
    q = queries(c, u, cuda, 92, noise=0.1)
    q[..., 0] = q[..., 0].abs() + 0.5
    finite = C.LayerCache(pc, cuda)   # what has weight: the reference is taken over it
    for f in R.FIELDS16 + R.FIELDS8 + ("n_bf16", "n_fp8"):
        getattr(finite, f).copy_(getattr(prefix, f))
    finite.k16[:, :n16 - 130], finite.v16[:, :n16 - 130] = prefix.k16[:, 130:], prefix.v16[:, 130:]
    finite.n_bf16.fill_(n16 - 130)
    few = R.cfg(prefixes * branches, hkv * G, hkv, d)
    ref = exact(few, finite, q[:few.batch], starts[:-1])
    o, ml = run(c, prefix, q, starts)
    check(few, (o[:-1], ml[:few.batch * hkv]), ref, 11)
    assert (o[-1] == 0).all() and (ml[few.batch * hkv:, :, 0] == float("-inf")).all() and (ml[few.batch * hkv:, :, 1] == 0).all()


@pytest.mark.parametrize("d,fmt,branches", [(128, "e4m3", 4), (64, "e5m2", 40)])
@pytest.mark.parametrize("up", [76, -76])
def test_range_of_the_values(cuda, d, fmt, branches, up):
    """Values around 2^76 and 2^-76 (n = 5000 tokens: 2^95 / n > 2^82) under logits just below the rise that moves the
    reference, 2^30 above where it starts and as far below."""
    n16, n8, hkv, G = 3000, 2000, 2, 4
    pc = R.cfg(1, hkv * G, hkv, d, n16, n8, fmt=fmt)
    prefix, u = heavy_prefix(pc, [n16], [n8], cuda, 100, heavy=0)
    g = gen(cuda, 101)
    fmax = 448.0 if fmt == "e4m3" else 57344.0
    level = 30 * math.log(2.0) * (1 if up > 0 else -1)
    for r in range(hkv):
        k = level / math.sqrt(d) * u[r] + 0.01 * torch.randn((n16 + n8, d), generator=g, device=cuda)
        prefix.k16[r] = k[:n16].bfloat16()
        s = k[n16:].abs().amax(-1) / fmax
        prefix.k8[r], prefix.sk[r] = (k[n16:] / s[:, None]).to(R.FP8[pc.quant_format]).view(torch.uint8), s
    prefix.v16.mul_(2.0 ** up)
    prefix.sv.mul_(2.0 ** up)
    c = R.cfg(branches, hkv * G, hkv, d)
    q = queries(c, u, cuda, 102, noise=0.01)
    ref = exact(c, prefix, q, [0, branches])
    check(c, run(c, prefix, q), ref, 79)


@pytest.mark.parametrize("d,G,prefixes,branches", [(128, 4, 32, 1), (64, 1, 20, 6), (64, 4, 20, 50)])
def test_nan_and_infinite_queries_in_long_runs(cuda, d, G, prefixes, branches):
    """Rows of NaN and infinite queries while the reference of their neighbours moves: they are NaN where the softmax
    is, and the others' bits stay."""
    hkv = 8
    prefix, u = rising_prefix(R.cfg(prefixes, hkv * G, hkv, d, 515, 509, fmt="e4m3"), cuda, 110)
    c = R.cfg(prefixes * branches, hkv * G, hkv, d)
    starts = [branches * i for i in range(prefixes + 1)]
    q = queries(c, u, cuda, 111, noise=0.1)
    clean, clean_ml = run(c, prefix, q, starts)
    hit = torch.zeros((c.batch, c.hq), dtype=torch.bool, device=cuda)
    for i in range(0, c.batch, 5):
        q[i, i % c.hq, 3] = float("nan")
        q[i, (i + 3) % c.hq] = float("inf") if i % 2 else float("-inf")
        hit[i, [i % c.hq, (i + 3) % c.hq]] = True
    o, ml = run(c, prefix, q, starts)
    assert torch.isnan(o[hit]).all()
    assert torch.equal(o[~hit], clean[~hit])
    rest = ~hit.view(c.batch * hkv, G)
    assert torch.equal(ml[:, :G][rest], clean_ml[:, :G][rest])
    assert int(prefix.status) == 0
