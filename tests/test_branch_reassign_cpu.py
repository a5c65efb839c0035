"""arkv_branch_reassign refuses bad arguments before any launch (no CUDA device is touched), and the row
capacities that the header gives for a branch's own tokens hold every count it can reach."""
import math

import pytest

from mixed_precision_kv_arkv_b200 import abi, build

P = 1 << 20   # a well aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def cfg(**kw):
    base = dict(batch=3, hq=8, hkv=2, head_dim=64, window=64, n_obs=64, gamma=1.0, budget_frac=0.25,
                cap_bf16=1000, cap_fp8=900, quant_format=abi.ARKV_FMT_E4M3, early_start=0)
    base.update(kw)
    return abi.arkv_cfg(*[base[n] for n, _ in abi.arkv_cfg._fields_])


def cache(at=1):
    return abi.arkv_layer_cache(*[4096 * (i + at) for i in range(15)])


@pytest.mark.parametrize("bad", [
    dict(cfg=cfg(window=0)), dict(cfg=cfg(hq=6)), dict(cfg=cfg(head_dim=128)), dict(prefix_cfg=cfg(batch=2, gamma=-1.0)),
    dict(prefix_cfg=cfg(batch=2, hkv=4)), dict(step=-1), dict(r=1.5), dict(r=float("nan")), dict(ctx_len=None),
    dict(cache=abi.arkv_layer_cache()), dict(prefix=abi.arkv_layer_cache()), dict(branch_start=None),
    dict(branch_start=P + 2), dict(ws=None), dict(ws=P + 16), dict(ws_bytes=100)])
def test_refusals(bad):
    c = dict(cfg=cfg(), step=0, r=0.5, ctx_len=P, cache=cache(), prefix_cfg=cfg(batch=2), prefix=cache(100), branch_start=P,
             tier_dbg=None, ws=4 * P, ws_bytes=1 << 30, stream=None)
    assert abi.arkv_branch_reassign(**{**c, **bad}, check=False) == abi.ARKV_EINVAL
    assert "arkv_branch_reassign" in abi.arkv_last_error_string() or "cfg" in abi.arkv_last_error_string() \
        or "cache" in abi.arkv_last_error_string() or "workspace" in abi.arkv_last_error_string()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("beta", [0.1, 0.25, 0.6])
@pytest.mark.parametrize("r", [0.0, 0.05, 0.5, 0.95, 1.0])
def test_own_capacities_hold_every_count(d, beta, r):
    """The counts of a branch behind a prefix that was packed under the same budget, against
    arkv_row_capacity for the own tokens and 2 / budget_frac more."""
    W, interval = 16, 4
    count = lambda n, held: (lambda rb: max(0, math.floor(rb / (r * 4 * d + (1 - r) * (2 * d + 8)))))(
        beta * n * 4 * d - W * 4 * d - held)
    for n0 in list(range(math.ceil(W / beta), math.ceil(W / beta) + 60)) + [1000, 4097, 32768]:
        sel = count(n0, 0)
        if sel >= n0 - W:
            continue   # its length set its count
        n_o = math.floor(r * sel)
        held = (W + n_o) * 4 * d + (sel - n_o) * (2 * d + 8)
        for own in (W + 1, 50, 300, 2000):
            cap16, cap8 = abi.arkv_row_capacity(cfg(head_dim=d, window=W, budget_frac=beta), own + math.ceil(2 / beta), r, interval)
            mine = min(count(n0 + own, held), own - W)
            assert math.floor(r * mine) + W + interval <= cap16 and mine <= cap8, (n0, own)
