"""The tier reassignment of branches that share a prefix: the bytes of the prefix's kept tokens are
part of a branch's budget, as they would be of a copy's."""
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


def held_bytes(prefix, row):
    d = prefix.cfg.head_dim
    return int(prefix.n_bf16[row]) * 4 * d + int(prefix.n_fp8[row]) * (2 * d + 8)


def selected(beta, n_t, r, d, w, held, cand):
    """(n_sel, n_o) of a row whose prefix keeps `held` bytes; the operations in the library's order."""
    rb = beta * n_t * (4.0 * d) - w * (4.0 * d) - held
    n_sel = min(max(0, math.floor(rb / (r * 4.0 * d + (1 - r) * (2.0 * d + 8.0)))) if rb > 0 else 0, cand)
    return n_sel, math.floor(r * n_sel)


def prompt_cache(c, ctx, n, r, dev, seed):
    """`len(ctx)` random prompts, scored and packed."""
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()
    k, v, q_obs = rn(c.batch, c.hkv, n, c.head_dim), rn(c.batch, c.hkv, n, c.head_dim), rn(c.batch, c.hq, c.n_obs, c.head_dim)
    prompt = C.LayerCache(c, dev)
    ws = C.Workspace(abi.arkv_workspace_bytes(c, abi.ARKV_WS_PREFILL, n), dev)
    f64 = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)
    stats, mu0, m20 = f64(3), f64(c.batch * c.hkv, n), f64(c.batch * c.hkv, n)
    s = C.stream_ptr()
    abi.arkv_prefill_stats(c, q_obs.data_ptr(), k.data_ptr(), n, ctx.data_ptr(), stats.data_ptr(), None, mu0.data_ptr(),
                           m20.data_ptr(), ws.ptr, ws.nbytes, s)
    abi.arkv_quantize_pack(c, r, k.data_ptr(), v.data_ptr(), n, ctx.data_ptr(), mu0.data_ptr(), m20.data_ptr(), prompt.c,
                           None, ws.ptr, ws.nbytes, s)
    torch.cuda.synchronize()
    return prompt


@pytest.mark.parametrize("d,fmt,r", [(64, "e4m3", 0.5), (128, "e5m2", 0.3)])
def test_branches_stay_within_the_budget_of_their_context(cuda, d, fmt, r):
    """80 steps of five branches (two of one prompt, two of another, one without) whose caches are sized for their
    own tokens: after every reassignment a row keeps its window and the budget's count, no token is dropped for
    want of room, and with the prefix's bytes a branch is within budget_frac of its whole context."""
    hq, hkv, W, beta, interval, steps = 8, 2, 8, 0.25, 4, 80
    ctx = torch.tensor([600, 517], dtype=torch.int32, device=cuda)
    prompt = prompt_cache(C.make_cfg(2, hq, hkv, d, W, W, 1.0, beta, 300, 300, fmt), ctx, 600, r, cuda, 3)
    starts, of = [0, 2, 4], [0, 0, 1, 1, None]
    B = len(of)
    bctx = torch.tensor([600, 600, 517, 517, 0], dtype=torch.int32, device=cuda)
    r = float(torch.tensor(r, dtype=torch.float32))
    size = C.make_cfg(B, hq, hkv, d, W, W, 1.0, beta, 1, 1, fmt)
    cap16, cap8 = abi.arkv_row_capacity(size, steps + math.ceil(2 / beta), r, interval)
    assert cap16 < steps // 2   # (own tokens have to be evicted for the branches to fit)
    st = C.new_layer_state(C.make_cfg(B, hq, hkv, d, W, W, 1.0, beta, cap16, cap8, fmt), r, cuda)
    sp = C.new_shared_prefix(st.cfg, prompt, starts)
    g = torch.Generator(device=cuda).manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=g, device=cuda).bfloat16()
    o_own, o = torch.zeros((B, hq, d), device=cuda), torch.zeros((B, hq, d), dtype=torch.bfloat16, device=cuda)
    live = [0] * (B * hkv)
    for t in range(steps):
        C.branch_step(st, sp, t, rn(B, hq, d), rn(B, hkv, d), rn(B, hkv, d), bctx, o_own, o, interval)
        torch.cuda.synchronize()
        n16, n8 = st.cache.n_bf16.tolist(), st.cache.n_fp8.tolist()
        for row in range(B * hkv):
            b, h = divmod(row, hkv)
            live[row] += 1
            held = 0 if of[b] is None else held_bytes(prompt, of[b] * hkv + h)
            n_t = int(bctx[b]) + t + 1
            if (t + 1) % interval == 0:
                cand = max(live[row] - W, 0)
                live[row] -= cand - selected(beta, n_t, r, d, W, held, cand)[0]
                mine = n16[row] * 4 * d + n8[row] * (2 * d + 8)
                assert held + mine <= max(beta * n_t * 4 * d, held + W * 4 * d), (t, row)
            assert n16[row] + n8[row] == live[row], (t, row)
        assert torch.isfinite(o).all()
    assert int(st.cache.status) == 0
    assert max(live) < steps // 2


def branch_rows(c, n0, step, dev, seed):
    """Random own caches of branches whose W newest tokens are in the bf16 segment; the other tokens have
    positions of their own before them."""
    n16, n8 = [40 + 7 * b % 25 for b in range(c.batch)], [50 - 5 * b % 30 for b in range(c.batch)]
    cache = R.random_cache(c, n16, n8, dev, seed)
    g = torch.Generator().manual_seed(seed)
    for row in range(c.batch * c.hkv):
        a, b = n16[row // c.hkv], n8[row // c.hkv]
        pos = torch.randperm(n0 + step + 1 - c.window, generator=g)[:a + b - c.window].int()
        cache.pos16[row, :c.window] = torch.arange(n0 + step + 1 - c.window, n0 + step + 1, dtype=torch.int32)
        cache.pos16[row, c.window:a] = pos[:a - c.window]
        cache.pos8[row, :b] = pos[a - c.window:]
    return cache


@pytest.mark.parametrize("d,r", [(64, 0.5), (128, 0.3), (64, 0.0), (128, 1.0)])
def test_branch_reassign_ranks_within_the_budget_left(cuda, d, r):
    """Tiers of every slot against the ranking by score cut at the counts that the prefix's bytes leave, for
    prefixes that leave all, some and nothing of the budget, an empty one, and branches without one."""
    import numpy as np
    from oracle import arkv as A
    hq, hkv, W, n0, step, beta = 8, 4, 6, 900, 4, 0.25
    pre16, pre8 = [0, 30, 170, 130, 220], [0, 40, 30, 100, 200]
    starts = [1, 2, 4, 4, 6, 7]                      # branches 0 and 7 without; nobody has the third
    pc = R.cfg(5, hq, hkv, d, 225, 210)
    prefix = R.random_cache(pc, pre16, pre8, cuda, 5)
    c = C.make_cfg(8, hq, hkv, d, W, 16, 1.5, beta, 70, 130, "e4m3")
    cache = branch_rows(c, n0, step, cuda, 6)
    of = [None, 0, 1, 1, 3, 3, 4, None]
    ctx = torch.full((8,), n0, dtype=torch.int32, device=cuda)
    before = {f: getattr(cache, f).clone() for f in ("pos16", "mu16", "m2_16", "pos8", "mu8", "m2_8", "n_bf16", "n_fp8")}
    tiers = torch.full((8 * hkv, 200), 9, dtype=torch.uint8, device=cuda)
    ws = C.Workspace(abi.arkv_workspace_bytes(c, abi.ARKV_WS_REASSIGN), cuda)
    bs = torch.tensor(starts, dtype=torch.int32, device=cuda)
    r = float(np.float32(r))
    abi.arkv_branch_reassign(c, step, r, ctx.data_ptr(), cache.c, pc, prefix.c, bs.data_ptr(), tiers.data_ptr(), ws.ptr,
                             ws.nbytes, C.stream_ptr())
    torch.cuda.synchronize()
    seen = set()
    for row in range(8 * hkv):
        b, h = divmod(row, hkv)
        a, n8 = int(before["n_bf16"][row]), int(before["n_fp8"][row])
        cat = lambda x, y: np.concatenate([before[x][row, :a].cpu().numpy(), before[y][row, :n8].cpu().numpy()])
        pos, mu, m2 = cat("pos16", "pos8"), cat("mu16", "mu8"), cat("m2_16", "m2_8")
        count = np.where(pos < n0, np.minimum(16, n0 - pos) + step + 1, step - (pos - n0) + 1)
        orig = np.arange(a + n8) < a
        cand = ~(orig & (pos >= n0 + step + 1 - W))
        held = 0 if of[b] is None else held_bytes(prefix, of[b] * hkv + h)
        n_sel, n_o = selected(beta, n0 + step + 1, r, d, W, held, int(cand.sum()))
        want = np.full(a + n8, A.ORIGINAL, np.int8)
        want[cand] = A.assign_tiers(A.heavy_hitter_score(mu, m2, count, 1.5)[cand], pos[cand], orig[cand], n_sel, n_o)[0]
        got = np.concatenate([tiers[row, :a].cpu().numpy(), tiers[row, 70:70 + n8].cpu().numpy()])
        assert (got == want).all(), (row, n_sel, n_o)
        seen.add("all" if n_sel == cand.sum() else "none" if n_sel == 0 else "some")
    # with r = 0 what the fourth prefix leaves, 9504 bytes, is 69 FP8 tokens: all of its branches'
    assert seen == ({"all", "some", "none"} if r > 0 else {"all", "none"}) and int(cache.status) == 0


def test_branch_reassign_without_a_prefix_is_reassign(cuda):
    """Empty prefixes and branches of no prefix: the bits of arkv_reassign."""
    c = C.make_cfg(5, 8, 2, 64, 6, 16, 1.0, 0.05, 70, 130, "e5m2")
    pc = R.cfg(2, 8, 2, 64, 20, 20)
    prefix = R.random_cache(pc, [0, 20], [0, 20], cuda, 7)
    ctx = torch.full((5,), 700, dtype=torch.int32, device=cuda)
    ws = C.Workspace(abi.arkv_workspace_bytes(c, abi.ARKV_WS_REASSIGN), cuda)
    bs = torch.tensor([1, 4, 4], dtype=torch.int32, device=cuda)
    a, b = branch_rows(c, 700, 3, cuda, 8), branch_rows(c, 700, 3, cuda, 8)
    abi.arkv_reassign(c, 3, 0.5, ctx.data_ptr(), a.c, None, ws.ptr, ws.nbytes, C.stream_ptr())
    abi.arkv_branch_reassign(c, 3, 0.5, ctx.data_ptr(), b.c, pc, prefix.c, bs.data_ptr(), None, ws.ptr, ws.nbytes, C.stream_ptr())
    torch.cuda.synchronize()
    assert int(a.n_bf16[0] + a.n_fp8[0]) < 90   # (some were evicted)
    for f, _ in abi.arkv_layer_cache._fields_:
        x, y = getattr(a, f), getattr(b, f)
        assert torch.equal(x.view(torch.uint8) if x.dtype != torch.int32 else x, y.view(torch.uint8) if y.dtype != torch.int32 else y), f
