"""Sizes past what the kernels index are host-side argument errors (ARKV_EINVAL) of the fork and the
shared-prefix attention, and have no workspace; just below them a workspace is given.  No CUDA device is
touched."""
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


PAST = [   # branches, prefixes
    (dict(batch=1 << 22), dict(batch=2, cap_bf16=1 << 20, cap_fp8=1 << 20)),     # places of the list of tiles
    (dict(batch=1 << 30, hq=4, hkv=4), dict(batch=1, hq=4, hkv=4, cap_bf16=1, cap_fp8=1)),   # heads of all branches
    (dict(batch=1 << 26), dict(batch=1, cap_bf16=1, cap_fp8=1)),                 # branches times rows of a unit
    (dict(), dict(batch=1 << 30, cap_bf16=1, cap_fp8=1)),                        # rows past 31 bits
    (dict(), dict(batch=1 << 10, cap_bf16=1 << 20)),                             # slots past 31 bits
]


@pytest.mark.parametrize("branches,prefixes", PAST)
def test_prefix_sizes(branches, prefixes):
    c, pc = cfg(**branches), cfg(**prefixes)
    assert abi.arkv_prefix_workspace_bytes(c, pc) == 0
    assert abi.arkv_prefix_attn(c, pc, P, cache(), P, None, None, 2 * P, None, 4 * P, 1 << 50, None, check=False) == abi.ARKV_EINVAL
    assert "31 bits" in abi.arkv_last_error_string()


def test_prefix_sizes_below():
    for branches, prefixes in ((dict(batch=1 << 20), dict(batch=2, cap_bf16=1 << 20, cap_fp8=1 << 20)),
                               (dict(batch=1 << 24), dict(batch=1, cap_bf16=1, cap_fp8=1)),
                               (dict(), dict(batch=1 << 10, cap_bf16=1 << 19))):
        assert abi.arkv_prefix_workspace_bytes(cfg(**branches), cfg(**prefixes)) > 0


@pytest.mark.parametrize("dst,src", [(dict(batch=1 << 30), dict()), (dict(), dict(batch=1 << 30))])
def test_fork_sizes(dst, src):
    assert abi.arkv_cache_fork(cfg(**dst), cache(1), cfg(**src), cache(100), P, None, check=False) == abi.ARKV_EINVAL
    assert "31 bits" in abi.arkv_last_error_string()
