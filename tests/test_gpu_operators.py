"""GPU checks of arkv_qk_norm_rope, arkv_cache_fork and arkv_prefix_attn against plain 64-bit
forms (tests/plain_ops.py holds those and the rounding bounds), and of the calls together:
a prompt prepared, packed, shared by branches or forked for them, and decoded."""
from __future__ import annotations

import math

import numpy as np
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


def bits(t):
    """A view that compares NaN patterns too."""
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


# ------------------------------------------------------------------ norm and rotation
ROPE_CASES = [
    # batch, tokens, hq, hkv, D, rot, interleaved, norm, ragged, extra stride, pos0
    (4, 1, 32, 8, 128, 128, 0, True, False, 0, 131071),
    (1, 1, 1, 1, 64, 64, 0, False, False, 0, 0),
    (3, 1, 3, 1, 128, 64, 0, True, False, 8, 2000000000),
    (2, 1, 8, 2, 64, 50, 0, True, False, 0, 7),          # pairs that straddle vectors
    (2, 37, 6, 2, 128, 126, 0, True, True, 24, 5),
    (3, 65, 4, 4, 64, 32, 1, True, True, 0, 0),
    (2, 33, 8, 2, 128, 128, 1, False, True, 0, 90000),
    (2, 19, 8, 2, 64, 0, 0, True, False, 0, 0),
    (1, 300, 8, 8, 64, 2, 0, False, False, 0, 0),
    (5, 130, 12, 3, 128, 16, 0, True, True, 0, 0),
    (150, 1, 8, 2, 128, 128, 0, True, False, 0, 9999),
    (3, 1001, 16, 4, 128, 128, 0, True, True, 0, 3),     # token counts a block's groups do not divide by
    (5, 1403, 16, 4, 64, 64, 1, True, True, 0, 11),
    (1, 8000, 16, 4, 64, 48, 0, True, False, 0, 0),
]


@pytest.mark.parametrize("batch,n,hq,hkv,d,rot,inter,norm,ragged,extra,at", ROPE_CASES)
def test_qk_norm_rope(cuda, batch, n, hq, hkv, d, rot, inter, norm, ragged, extra, at):
    g = gen(cuda, 1)
    n_obs, width = 7, (hq + 2 * hkv) * d
    c = R.cfg(batch, hq, hkv, d, n_obs=n_obs)
    qkv = torch.randn((batch * n, width + extra), generator=g, device=cuda).bfloat16()
    wq, wk = [(1 + 0.3 * torch.randn(d, generator=g, device=cuda)).bfloat16() if norm else None for _ in range(2)]
    freq = C.rope_frequencies(rot, 500000.0, cuda) if rot else None
    pos0 = torch.randint(max(0, at - 3), at + 1, (batch,), generator=g, device=cuda, dtype=torch.int32) if at else None
    length = None
    live = torch.full((batch,), n, device=cuda)
    if ragged:   # a whole one, an empty one, one past the end (clamped), shorter ones
        length = torch.tensor([n, 0, n + 9, n // 2, 3][:batch], dtype=torch.int32, device=cuda)
        live = length.long().clamp(max=n)
        for b in range(batch):   # padding rows are not read
            qkv.view(batch, n, -1)[b, int(live[b]):] = float("nan")
    stride = n + 3
    mk = lambda h, m: torch.full((batch, h, m, d), 7.0, dtype=torch.bfloat16, device=cuda)
    q, k, v, q_obs = mk(hq, stride), mk(hkv, stride), mk(hkv, stride), mk(hq, n_obs)
    step = 2 if at else 0
    C.qk_norm_rope(c, qkv, n, freq, k, v, q, q_obs, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=inter, pos0=pos0,
                   step=step, length=length)
    clean = torch.where(torch.isnan(qkv), torch.zeros_like(qkv), qkv)
    rq, rk, rv, bq, bk = R.qk_norm_rope(c, n, clean, pos0, step, live, wq, wk, 1e-5, freq, rot, inter)
    for b in range(batch):
        m = int(live[b])
        for got, ref, bound in ((q, rq, bq), (k, rk, bk)):
            err = (got[b, :, :m].double() - ref[b, :, :m]).abs()
            assert (err <= bound[b, :, :m]).all(), (b, float((err / (bound[b, :, :m] + 1e-30)).max()))
        assert torch.equal(v[b, :, :m].double(), rv[b, :, :m])
        for got in (q, k, v):   # padding and the room behind it stay as they were
            assert (got[b, :, m:] == 7.0).all()
        o = min(m, n_obs)
        assert torch.equal(q_obs[b, :, n_obs - o:], q[b, :, m - o:m])
        assert (q_obs[b, :, :n_obs - o] == 7.0).all()
    k2, v2 = mk(hkv, stride), mk(hkv, stride)   # without the nullable outputs: the same keys and values
    C.qk_norm_rope(c, qkv, n, freq, k2, v2, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=inter, pos0=pos0, step=step,
                   length=length)
    assert torch.equal(bits(k), bits(k2)) and torch.equal(bits(v), bits(v2))


def test_qk_norm_rope_zero_and_huge_heads(cuda):
    """A head of zeros stays zero (eps keeps the norm finite); large values do not overflow the norm."""
    c = R.cfg(1, 2, 1, 64)
    qkv = torch.zeros((1, 4 * 64), dtype=torch.bfloat16, device=cuda)
    qkv[0, 64:128] = 2.0 ** 60
    one = torch.ones(64, dtype=torch.bfloat16, device=cuda)
    mk = lambda h: torch.empty((1, h, 1, 64), dtype=torch.bfloat16, device=cuda)
    q, k, v = mk(2), mk(1), mk(1)
    C.qk_norm_rope(c, qkv, 1, None, k, v, q, q_weight=one, k_weight=one)
    assert (q[0, 0] == 0).all() and (k == 0).all() and (q[0, 1] == 1).all()


def test_qk_norm_rope_wrapper_refusals(cuda):
    c = R.cfg(2, 2, 1, 64)
    qkv = torch.zeros((2, 256), dtype=torch.bfloat16, device=cuda)
    k = torch.zeros((2, 1, 1, 64), dtype=torch.bfloat16, device=cuda)
    for bad in (dict(qkv=qkv[:1]), dict(qkv=qkv.float()), dict(k=k[:, :, :, :32]), dict(v=k.float()),
                dict(pos0=torch.zeros(2, device=cuda)), dict(q_obs=k)):
        a = dict(dict(qkv=qkv, n_tok=1, freq=None, k=k, v=k.clone()), **bad)
        with pytest.raises(ValueError):
            C.qk_norm_rope(c, a.pop("qkv"), a.pop("n_tok"), a.pop("freq"), a.pop("k"), a.pop("v"), **a)


# ------------------------------------------------------------------ fork
def clone(cache, dev):
    out = C.LayerCache(cache.cfg, dev)
    for name, _ in abi.arkv_layer_cache._fields_:
        getattr(out, name).copy_(getattr(cache, name))
    return out


def forked(dst, src, seqs, in_place=False):
    """The buffers arkv_cache_fork leaves, by plain copies; and the status bits."""
    hkv = dst.cfg.hkv
    want = {n: getattr(dst, n).clone() for n, _ in abi.arkv_layer_cache._fields_}
    status = 0
    for b, s in enumerate(seqs):
        rows = slice(b * hkv, (b + 1) * hkv)
        if s == abi.ARKV_SEQ_KEEP:
            continue
        if s == abi.ARKV_SEQ_FREE:
            want["n_bf16"][rows], want["n_fp8"][rows] = 0, 0
            continue
        if not 0 <= s < src.cfg.batch or (in_place and seqs[s] not in (s, abi.ARKV_SEQ_KEEP)):
            status |= abi.ARKV_STATUS_BAD_FORK
            continue
        for g in range(hkv):
            for fields, n_name, cap, bit in ((R.FIELDS16, "n_bf16", dst.cfg.cap_bf16, abi.ARKV_STATUS_BF16_FULL),
                                             (R.FIELDS8, "n_fp8", dst.cfg.cap_fp8, abi.ARKV_STATUS_FP8_FULL)):
                n = int(getattr(src, n_name)[s * hkv + g])
                status |= bit if n > cap else 0
                n = min(n, cap)
                for f in fields:
                    want[f][b * hkv + g, :n] = getattr(src, f)[s * hkv + g, :n]
                want[n_name][b * hkv + g] = n
    return want, status


def assert_fork(dst, src, seqs, cuda, in_place=False, stream=None):
    want, status = forked(dst, src, seqs, in_place)
    C.fork(dst, src, torch.tensor(seqs, dtype=torch.int32, device=cuda), stream=stream)
    torch.cuda.synchronize()
    for name, x in want.items():
        if name != "status":
            assert torch.equal(bits(getattr(dst, name)), bits(x)), name
    assert int(dst.status) == status


@pytest.mark.parametrize("hkv,d,cap,dcap,n16,n8,seqs", [
    (1, 64, (1, 1), (1, 1), [1], [0], [0]),
    (2, 64, (40, 33), (40, 33), [40, 0], [33, 7], [1, 0, 0, 1, 1]),
    (2, 128, (301, 267), (303, 262), [301, 5], [255, 1], [0, 1, abi.ARKV_SEQ_KEEP, 0, abi.ARKV_SEQ_FREE]),   # odd strides
    (3, 128, (300, 700), (129, 650), [300, 100], [700, 0], [0, 1, 0]),                 # smaller capacities: cut, flagged
    (2, 64, (20, 20), (20, 20), [7, 9], [3, 20], [5, -3, 1, 2, 0]),                    # sources out of range
    (8, 128, (1500, 900), (1500, 900), [1500], [900], [0] * 40),                       # one source, many copies
])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_fork(cuda, hkv, d, cap, dcap, n16, n8, seqs, fmt):
    src = R.random_cache(R.cfg(len(n16), hkv, hkv, d, *cap, fmt=fmt), n16, n8, cuda, 3)
    keep = clone(src, cuda)
    dc = R.cfg(len(seqs), hkv, hkv, d, *dcap, fmt=fmt)
    dst = R.random_cache(dc, [1] * len(seqs), [1] * len(seqs), cuda, 4)
    assert_fork(dst, src, seqs, cuda)
    for name, _ in abi.arkv_layer_cache._fields_:
        assert torch.equal(bits(getattr(src, name)), bits(getattr(keep, name))), name


@pytest.mark.parametrize("seqs", [
    [0, 0, 2, 2, 4, 4], [abi.ARKV_SEQ_KEEP, 0, 0, 0, abi.ARKV_SEQ_FREE, 0],
    [0, 1, 2, 3, 4, 5],
    [1, 0, 2, 3, 4, 4],      # a swap: both sources lose their state, so both stay
    [1, 2, 2, 2, 9, 5],      # a chain: only the copies of 2 go through
    [abi.ARKV_SEQ_FREE, 0, 2, 2, 4, 5],   # the freed sequence is no source
])
def test_fork_in_place(cuda, seqs):
    cache = R.random_cache(R.cfg(6, 4, 4, 64, 150, 131), [150, 0, 77, 1, 128, 20], [0, 131, 64, 2, 3, 9], cuda, 5)
    assert_fork(cache, cache, seqs, cuda, in_place=True)


# ------------------------------------------------------------------ shared prefix
def own_part(c, cuda, seed, level):
    g = gen(cuda, seed)
    o = torch.randn((c.batch, c.hq, c.head_dim), generator=g, device=cuda)
    ml = torch.zeros((c.batch * c.hkv, 4, 2), device=cuda)
    ml[..., 0] = level + 10 * torch.randn((c.batch * c.hkv, 4), generator=g, device=cuda)
    ml[..., 1] = 1 + 20 * torch.rand((c.batch * c.hkv, 4), generator=g, device=cuda)
    return o, ml


def run_prefix(c, prefix, q, starts, o_own=None, ml_own=None, stream=None, sp=None, with_ml=True):
    sp = sp or C.new_shared_prefix(c, prefix, starts)
    o = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device=q.device)
    ml = torch.full((c.batch * c.hkv, 4, 2), 5.0, device=q.device) if with_ml else None
    ptr = C._ptr
    abi.arkv_prefix_attn(c, prefix.cfg, ptr(q), prefix.c, ptr(sp.branch_start), ptr(o_own), ptr(ml_own), ptr(o), ptr(ml),
                         sp.ws.ptr, sp.ws.nbytes, C.stream_ptr(stream))
    return o, ml


PREFIX_CASES = [
    # hq, hkv, D, fmt, n16, n8 (by prefix), starts (None: one prefix for every branch), branches
    (4, 1, 128, "e4m3", [1], [0], None, 1),
    (1, 1, 64, "e4m3", [0], [1], None, 1),
    (2, 1, 64, "e5m2", [127], [129], None, 3),
    (8, 2, 64, "e4m3", [128], [128], None, 5),
    (8, 2, 128, "e5m2", [129], [0], None, 2),
    (8, 2, 128, "e4m3", [0], [257], None, 33),
    (3, 1, 128, "e4m3", [600], [515], None, 43),             # groups of three, one branch past a tile of them
    (6, 2, 64, "e5m2", [333], [1], None, 85),
    (4, 4, 128, "e4m3", [1000], [700], None, 130),           # one query a key head, past 128 branches
    (4, 1, 64, "e4m3", [300], [1000], None, 70),             # 280 query rows a key head
    (32, 8, 128, "e4m3", [1900], [1500], None, 4),
    (32, 8, 128, "e5m2", [3000], [2500], None, 40),
    (8, 2, 128, "e4m3", [200, 0, 5, 400], [100, 0, 0, 900], [1, 4, 4, 5, 12], 14),   # without: 0, 12, 13; an empty group
    (12, 4, 128, "e5m2", [1, 260, 40], [1, 10, 600], [0, 1, 30, 36], 36),
    (16, 8, 64, "e4m3", [(17 * i) % 300 for i in range(40)], [(71 * i) % 290 for i in range(40)],
     [2 * i for i in range(41)], 80),                        # more rows than CTAs
]


@pytest.mark.parametrize("hq,hkv,d,fmt,n16,n8,starts,branches", PREFIX_CASES)
def test_prefix_attn(cuda, hq, hkv, d, fmt, n16, n8, starts, branches):
    pc = R.cfg(len(n16), hq, hkv, d, max(n16) + 5, max(n8) + 3, fmt=fmt)
    prefix = R.random_cache(pc, n16, n8, cuda, 6)
    c = R.cfg(branches, hq, hkv, d)
    q = torch.randn((branches, hq, d), generator=gen(cuda, 7), device=cuda).bfloat16()
    span = starts or [0, branches]
    o_own, ml_own = own_part(c, cuda, 8, 2.5 * d ** 0.5)
    ml_own[1 % ml_own.shape[0], :, 1] = 0.0       # heads without own tokens
    ml_own[1 % ml_own.shape[0], :, 0] = float("-inf")
    o_own.view(branches * hkv, hq // hkv, d)[1 % ml_own.shape[0]] = 0.0
    o, ml = run_prefix(c, prefix, q, starts, o_own, ml_own)
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, span, o_own, ml_own))
    assert (ml[:, hq // hkv:] == 5.0).all()       # the padded heads stay as they were
    o, ml = run_prefix(c, prefix, q, starts)      # the prefix alone
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, span))
    o2, _ = run_prefix(c, prefix, q, starts, with_ml=False)
    assert torch.equal(o, o2)                     # and again: the same bits
    assert int(prefix.status) == 0


@pytest.mark.parametrize("d,fmt", [(64, "e4m3"), (128, "e5m2"), (128, "e4m3")])
def test_prefix_attn_sharp_and_far_logits(cuda, d, fmt):
    """Logits that grow along the prefix (the softmax reference keeps moving), one that dwarfs the
    others, FP8 scales from 2^-40 to 2^10."""
    n16, n8, hkv, G, B = 700, 650, 2, 4, 20
    pc = R.cfg(1, hkv * G, hkv, d, n16, n8, fmt=fmt)
    prefix = R.random_cache(pc, [n16], [n8], cuda, 9, poison=False)
    u = torch.randn((hkv, 1, d), generator=gen(cuda, 10), device=cuda)
    ramp = torch.linspace(-3, 3, n16, device=cuda)[None, :, None]
    prefix.k16.copy_((prefix.k16.float() * 0.3 + ramp * u).bfloat16())
    prefix.k16[0, 350] *= 3
    prefix.sk *= torch.exp2(torch.linspace(-40, 6, n8, device=cuda))
    prefix.sv *= torch.exp2(torch.linspace(10, -30, n8, device=cuda))
    c = R.cfg(B, hkv * G, hkv, d)
    q = (torch.randn((B, hkv * G, d), generator=gen(cuda, 11), device=cuda)
         + 1.5 * u.repeat_interleave(G, 0).view(1, hkv * G, d)).bfloat16()
    o, ml = run_prefix(c, prefix, q, None)
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, [0, B]))


def test_prefix_attn_counts_past_capacity_and_odd_starts(cuda):
    """Counts are clamped to the capacities, branch_start to 0..batch and to an order."""
    pc = R.cfg(3, 4, 2, 64, 150, 140)
    prefix = R.random_cache(pc, [150, 60, 9], [140, 9, 140], cuda, 12)
    c = R.cfg(9, 4, 2, 64)
    q = torch.randn((9, 4, 64), generator=gen(cuda, 13), device=cuda).bfloat16()
    prefix.n_bf16[0], prefix.n_fp8[1], prefix.n_fp8[4] = 151, 1 << 30, -5
    prefix.n_fp8[0], prefix.n_fp8[1] = 140, 1 << 30
    o, ml = run_prefix(c, prefix, q, [-4, 3, 5, 90])
    saved = prefix.n_fp8.clone()
    prefix.n_fp8[4] = 0
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, [0, 3, 5, 9]))
    prefix.n_fp8.copy_(saved)


def test_prefix_attn_nan_stays_in_its_branch(cuda):
    pc = R.cfg(1, 8, 2, 128, 300, 300)
    prefix = R.random_cache(pc, [300], [300], cuda, 14)
    c = R.cfg(40, 8, 2, 128)
    q = torch.randn((40, 8, 128), generator=gen(cuda, 15), device=cuda).bfloat16()
    clean, _ = run_prefix(c, prefix, q, None)
    q[7, 3, 5], q[22] = float("nan"), float("inf")
    o, _ = run_prefix(c, prefix, q, None)
    assert torch.isnan(o[7, 3]).all()
    hit = torch.zeros((40, 8), dtype=torch.bool, device=cuda)
    hit[7, 3], hit[22] = True, True
    assert torch.equal(o[~hit], clean[~hit])


# ------------------------------------------------------------------ streams and graphs
def test_on_another_stream_and_in_a_graph(cuda):
    """The three calls on a side stream, then captured into a graph and replayed on new inputs: the
    results of plain calls, bit for bit; two graphs share the workspace."""
    B, hq, hkv, d = 6, 8, 2, 128
    c = R.cfg(B, hq, hkv, d, 400, 300, early=True)
    pc = R.cfg(1, hq, hkv, d, 400, 300)
    prefix = R.random_cache(pc, [390], [280], cuda, 16)
    copies = C.LayerCache(c, cuda)
    sp = C.new_shared_prefix(c, prefix)
    qkv = torch.zeros((B, (hq + 2 * hkv) * d), dtype=torch.bfloat16, device=cuda)
    freq = C.rope_frequencies(d, 1e4, cuda)
    pos0 = torch.full((B,), 670, dtype=torch.int32, device=cuda)
    seqs = torch.tensor([0, abi.ARKV_SEQ_FREE, 0, 0, 0, 0], dtype=torch.int32, device=cuda)
    mk = lambda h: torch.zeros((B, h, 1, d), dtype=torch.bfloat16, device=cuda)
    q, k, v = mk(hq), mk(hkv), mk(hkv)
    o, ml = torch.zeros((B, hq, d), dtype=torch.bfloat16, device=cuda), torch.zeros((B * hkv, 4, 2), device=cuda)

    def calls(stream):
        C.qk_norm_rope(c, qkv, 1, freq, k, v, q, pos0=pos0, stream=stream)
        C.fork(copies, prefix, seqs, stream=stream)
        abi.arkv_prefix_attn(c, pc, q.data_ptr(), prefix.c, None, None, None, o.data_ptr(), ml.data_ptr(), sp.ws.ptr,
                             sp.ws.nbytes, C.stream_ptr(stream))

    def outputs():
        torch.cuda.synchronize()
        return [x.clone() for x in (q, k, v, o, ml, copies.k16, copies.v8, copies.n_bf16)]

    inputs = [torch.randn(qkv.shape, generator=gen(cuda, 20 + i), device=cuda).bfloat16() for i in range(3)]
    plain = []
    for x in inputs:
        qkv.copy_(x)
        calls(torch.cuda.current_stream())
        plain.append(outputs())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qkv.copy_(inputs[1])
    calls(side)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(outputs(), plain[1]))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            calls(side)
        graphs.append(gr)
    for i, gr in ((0, graphs[0]), (2, graphs[1]), (1, graphs[0])):
        qkv.copy_(inputs[i])
        torch.cuda.synchronize()
        for x in (o, ml, copies.k16):
            x.zero_()
        gr.replay()
        got = outputs()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got[:5], plain[i][:5]))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt,d,early", [("e4m3", 128, False), ("e5m2", 64, True)])
def test_shared_and_forked_prompts_decode_alike(cuda, fmt, d, early):
    """Two prompts are normalised, rotated, scored and packed; five branches decode from them twice: with
    the packed prompts shared (arkv_prefix_attn) and with a fork each (arkv_decode_attn on the copy).
    Outputs and the scores of the new tokens agree within the rounding of P and o to bf16 (each 2^-8
    of at most the largest |v|) and the score tolerance of the decode path."""
    hq, hkv, N, W, steps = 8, 2, 700, 32, 6
    g = gen(cuda, 30)
    pc = C.make_cfg(2, hq, hkv, d, W, W, 1.0, 0.4, 400, 400, fmt)
    ctx = torch.tensor([700, 655], dtype=torch.int32, device=cuda)
    qkv = torch.randn((2 * N, (hq + 2 * hkv) * d), generator=g, device=cuda).bfloat16()
    wq, wk = [(1 + 0.2 * torch.randn(d, generator=g, device=cuda)).bfloat16() for _ in range(2)]
    freq = C.rope_frequencies(d, 1e6, cuda)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=cuda)
    k, v, q_obs = z(2, hkv, N, d), z(2, hkv, N, d), z(2, hq, W, d)
    C.qk_norm_rope(pc, qkv, N, freq, k, v, None, q_obs, q_weight=wq, k_weight=wk, length=ctx)
    prompt = C.LayerCache(pc, cuda)
    ws = C.Workspace(abi.arkv_workspace_bytes(pc, abi.ARKV_WS_PREFILL, N), cuda)
    f64 = lambda *s: torch.zeros(s, dtype=torch.float64, device=cuda)
    stats, mu0, m20 = f64(3), f64(2 * hkv, N), f64(2 * hkv, N)
    st = C.stream_ptr()
    abi.arkv_prefill_stats(pc, q_obs.data_ptr(), k.data_ptr(), N, ctx.data_ptr(), stats.data_ptr(), None, mu0.data_ptr(),
                           m20.data_ptr(), ws.ptr, ws.nbytes, st)
    abi.arkv_quantize_pack(pc, 0.5, k.data_ptr(), v.data_ptr(), N, ctx.data_ptr(), mu0.data_ptr(), m20.data_ptr(),
                           prompt.c, None, ws.ptr, ws.nbytes, st)
    of = [0, 0, 1, 1, 1]
    B = len(of)
    bctx = ctx[torch.tensor(of, device=cuda)].contiguous()
    shared = C.new_layer_state(C.make_cfg(B, hq, hkv, d, W, W, 1.0, 0.4, 40, 40, fmt, early), 0.5, cuda)
    sp = C.new_shared_prefix(shared.cfg, prompt, [0, 2, 5])
    copies = C.new_layer_state(C.make_cfg(B, hq, hkv, d, W, W, 1.0, 0.4, 440, 400, fmt), 0.5, cuda)
    C.fork(copies.cache, prompt, torch.tensor(of, dtype=torch.int32, device=cuda))
    n0 = copies.cache.n_bf16.clone()
    o_own, o_ref = torch.zeros((B, hq, d), device=cuda), torch.zeros((B, hq, d), device=cuda)
    o = z(B, hq, d)
    q, kn, vn = z(B, hq, 1, d), z(B, hkv, 1, d), z(B, hkv, 1, d)
    vmax = float(max(v.abs().max(), 1.0))
    for t in range(steps):
        row = torch.randn((B, (hq + 2 * hkv) * d), generator=g, device=cuda).bfloat16()
        C.qk_norm_rope(shared.cfg, row, 1, freq, kn, vn, q, q_weight=wq, k_weight=wk, pos0=bctx, step=t)
        if early:
            torch.cuda.synchronize()
        C.branch_step(shared, sp, t, q, kn, vn, bctx, o_own, o, 1 << 30)
        torch.cuda.synchronize()
        C.decode_step(copies, t, q, kn, vn, bctx, o_ref, 1 << 30)
        torch.cuda.synchronize()
        vmax = max(vmax, float(vn.abs().max()))
        assert float((o.float() - o_ref).abs().max()) <= 2.0 ** -7 * vmax, t
    a, b = shared.cache, copies.cache
    assert (a.n_bf16 == steps).all() and (b.n_bf16 == n0 + steps).all()
    for r in range(B * hkv):
        i = slice(int(n0[r]), int(n0[r]) + steps)
        assert torch.equal(a.pos16[r, :steps], b.pos16[r, i]) and torch.equal(a.k16[r, :steps], b.k16[r, i])
        for f in ("mu16", "m2_16"):
            x, y = getattr(a, f)[r, :steps], getattr(b, f)[r, i]
            assert ((x - y).abs() <= 2e-5 * y.abs() + 1e-12).all(), (f, r)
    C.branch_step(shared, sp, steps, q, kn, vn, bctx, o_own, o, 1)       # with a reassignment
    torch.cuda.synchronize()
    assert torch.isfinite(o).all() and int(a.status) == 0 and int(prompt.status) == 0


# ------------------------------------------------------------------ corners
@pytest.mark.parametrize("d,rot,inter", [(128, 64, 0), (64, 50, 0), (128, 64, 1), (64, 0, 0)])
def test_qk_norm_rope_infinite_weight_stays_in_its_dimension(cuda, d, rot, inter):
    """An infinite weight of a dimension that is not rotated reaches that dimension alone."""
    c = R.cfg(2, 4, 1, d)
    qkv = torch.randn((2, 6 * d), generator=gen(cuda, 40), device=cuda).bfloat16()
    w = (1 + 0.1 * torch.randn(d, generator=gen(cuda, 41), device=cuda)).bfloat16()
    freq = C.rope_frequencies(rot, 1e4, cuda) if rot else None
    mk = lambda h: torch.empty((2, h, 1, d), dtype=torch.bfloat16, device=cuda)
    outs = []
    for last in (1.0, float("inf")):
        w[d - 3] = last
        q, k, v = mk(4), mk(1), mk(1)
        C.qk_norm_rope(c, qkv, 1, freq, k, v, q, q_weight=w, k_weight=w, interleaved=inter, step=5)
        outs.append(torch.cat([q, k], 1))
    others = [i for i in range(d) if i != d - 3]
    assert torch.equal(outs[0][..., others], outs[1][..., others])
    assert torch.isinf(outs[1][..., d - 3]).all()


def test_prefix_attn_of_empty_prefixes(cuda):
    """No prefix token anywhere: the own part comes through (one rounding to bf16), or zeros."""
    pc, c = R.cfg(2, 8, 2, 128, 20, 20), R.cfg(5, 8, 2, 128)
    prefix = R.random_cache(pc, [0, 0], [0, 0], cuda, 42)
    q = torch.randn((5, 8, 128), generator=gen(cuda, 43), device=cuda).bfloat16()
    o_own, ml_own = own_part(c, cuda, 44, 3.0)
    o, ml = run_prefix(c, prefix, q, [0, 2, 5], o_own, ml_own)
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, [0, 2, 5], o_own, ml_own))
    o, ml = run_prefix(c, prefix, q, [0, 2, 5])
    assert (o == 0).all() and (ml[..., 0] == float("-inf")).all() and (ml[..., 1] == 0).all()


@pytest.mark.parametrize("d,branches", [(64, 3), (128, 3), (128, 40)])
def test_prefix_attn_zero_scales(cuda, d, branches):
    """K and V scales of zero, the last live token's among them (its scale is what the columns
    past the end of a tile meet)."""
    prefix = R.random_cache(R.cfg(1, 8, 2, d, 70, 170), [70], [157], cuda, 45)
    prefix.sk[:, [3, 80, 156]] = 0.0
    prefix.sv[:, [4, 81, 156]] = 0.0
    c = R.cfg(branches, 8, 2, d)
    q = torch.randn((branches, 8, d), generator=gen(cuda, 46), device=cuda).bfloat16()
    o, ml = run_prefix(c, prefix, q, None)
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, [0, branches]))


def test_rows_past_31_bits(cuda):
    """A cache whose rows lie past 2^31 elements and bytes: forked in place, shared and read."""
    cap = 2200001
    cache = R.random_cache(R.cfg(2, 8, 4, 128, cap, cap + 7), [300, 5], [257, 9], cuda, 47)
    assert cache.k8.numel() > 2 ** 31 and cache.k16.numel() > 2 ** 31
    C.fork(cache, cache, torch.tensor([0, 0], dtype=torch.int32, device=cuda))
    small = C.LayerCache(R.cfg(1, 8, 4, 128, 400, 400), cuda)
    C.fork(small, cache, torch.tensor([1], dtype=torch.int32, device=cuda))
    for f, n in [(f, 300) for f in R.FIELDS16] + [(f, 257) for f in R.FIELDS8]:
        x = getattr(cache, f)
        assert torch.equal(bits(x[:4, :n]), bits(x[4:, :n])) and torch.equal(bits(x[4:, :n]), bits(getattr(small, f)[:, :n])), f
    c = R.cfg(5, 8, 4, 128)
    q = torch.randn((5, 8, 128), generator=gen(cuda, 48), device=cuda).bfloat16()
    o, ml = run_prefix(c, cache, q, [0, 2, 5])
    R.check_prefix(c, o, ml, R.prefix_attn(c, cache, q, [0, 2, 5]))


def test_calls_on_two_streams_at_once(cuda):
    """Calls on two streams, each with its workspace, and several on one workspace one after the
    other: the bits of calls made alone."""
    c, pc = R.cfg(36, 8, 2, 128), R.cfg(2, 8, 2, 128, 2000, 1500)
    prefix = R.random_cache(pc, [2000, 900], [1500, 1100], cuda, 49)
    starts = [0, 20, 36]
    qs = [torch.randn((36, 8, 128), generator=gen(cuda, 50 + i), device=cuda).bfloat16() for i in range(6)]
    alone = []
    for q in qs:
        alone.append(run_prefix(c, prefix, q, starts))
        torch.cuda.synchronize()
    sides = [(torch.cuda.Stream(), C.new_shared_prefix(c, prefix, starts)) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i, q in enumerate(qs):
        with torch.cuda.stream(sides[i % 2][0]):
            got.append(run_prefix(c, prefix, q, starts, sp=sides[i % 2][1]))
    torch.cuda.synchronize()
    for a, b in zip(got, alone):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert int(prefix.status) == 0


def test_many_small_prefixes(cuda):
    """More rows than a warp has lanes, most without branches or tokens."""
    P, hkv = 100, 4
    n16, n8 = [(i % 7 == 0) * (i + 1) for i in range(P)], [(i % 5 == 0) * 2 * i for i in range(P)]
    sizes = [(i % 3 == 0) * (1 + i % 4) for i in range(P)]
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + s)
    prefix = R.random_cache(R.cfg(P, 8, hkv, 64, 110, 210, fmt="e5m2"), n16, n8, cuda, 56)
    c = R.cfg(starts[-1], 8, hkv, 64)
    q = torch.randn((c.batch, 8, 64), generator=gen(cuda, 57), device=cuda).bfloat16()
    o_own, ml_own = own_part(c, cuda, 58, 1.0)
    o, ml = run_prefix(c, prefix, q, starts, o_own, ml_own)
    R.check_prefix(c, o, ml, R.prefix_attn(c, prefix, q, starts, o_own, ml_own))


@pytest.mark.parametrize("branches", [40, 1400])
def test_prefix_attn_runs_over_many_units(cuda, branches):
    """Runs that cross units, with every number of bf16 tiles between the FP8 tiles of one unit and
    of the next, for one and two tiles of rows."""
    P, hkv = 40, 2
    n16, n8 = [64 * (i % 13) + (i % 3) for i in range(P)], [64 * ((5 * i) % 17) + 1 for i in range(P)]
    starts = [branches * i // P for i in range(P + 1)]
    prefix = R.random_cache(R.cfg(P, 8, hkv, 128, 800, 1100), n16, n8, cuda, 60)
    c = R.cfg(branches, 8, hkv, 128)
    q = torch.randn((branches, 8, 128), generator=gen(cuda, 61), device=cuda).bfloat16()
    first, ml = run_prefix(c, prefix, q, starts)
    R.check_prefix(c, first, ml, R.prefix_attn(c, prefix, q, starts))
    for _ in range(20):
        assert torch.equal(run_prefix(c, prefix, q, starts)[0], first)
    assert int(prefix.status) == 0


def test_wrapper_refusals(cuda):
    prompt = C.LayerCache(R.cfg(1, 8, 2, 64, 10, 10), cuda)
    c = C.make_cfg(2, 8, 2, 64, 4, 4, 1.0, 0.5, 20, 20, "e4m3")
    with pytest.raises(ValueError):
        C.new_shared_prefix(C.make_cfg(2, 8, 2, 128, 4, 4, 1.0, 0.5, 20, 20, "e4m3"), prompt)
    with pytest.raises(ValueError):
        C.new_shared_prefix(c, prompt, [0, 1, 2])
    st, sp = C.new_layer_state(c, 0.5, cuda), C.new_shared_prefix(c, prompt)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device=cuda)
    a = dict(q=z(2, 8, 1, 64), k_new=z(2, 2, 1, 64), v_new=z(2, 2, 1, 64), ctx_len=z(2, dt=torch.int32),
             o_own=z(2, 8, 64, dt=torch.float32), o=z(2, 8, 64))
    for bad in (dict(o=a["o_own"]), dict(o_own=a["o"]), dict(q=a["o_own"]), dict(ctx_len=z(2, dt=torch.int64)),
                dict(k_new=z(2, 2, 64, 2).transpose(2, 3)[:, :, :1])):
        with pytest.raises(ValueError):
            C.branch_step(st, sp, 0, **{**a, **bad}, reassign_interval=100)
    with pytest.raises(ValueError):
        C.fork(st.cache, prompt, torch.zeros(2, device=cuda))
