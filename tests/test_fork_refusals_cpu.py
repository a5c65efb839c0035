"""arkv_cache_fork between caches that cannot be forked into one another is refused before any launch (no CUDA
device is touched): other observation counts, and caches that share some of their buffers."""
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


def cache(*shared):
    """A cache whose buffers `shared` (by place) are those of every other such cache."""
    cache.next += 100
    return abi.arkv_layer_cache(*[4096 * (i + 1 if i in shared else i + cache.next) for i in range(15)])


cache.next = 0


def test_another_count_of_observations():
    """The scores' counts are a function of n_obs: a copy could not go on from there."""
    assert abi.arkv_cache_fork(cfg(n_obs=16), cache(), cfg(), cache(), P, None, check=False) == abi.ARKV_EINVAL
    assert "n_obs" in abi.arkv_last_error_string()


@pytest.mark.parametrize("shared", [(0,), (2,), (12,), (13,), tuple(range(13)), tuple(range(1, 14)), (0, 1, 5, 6)])
def test_some_buffers_shared(shared):
    """Neither one cache nor two: every buffer is the same, or none."""
    assert abi.arkv_cache_fork(cfg(), cache(*shared), cfg(), cache(*shared), P, None, check=False) == abi.ARKV_EINVAL
    assert "share no buffer" in abi.arkv_last_error_string()


@pytest.mark.parametrize("other", [dict(batch=2), dict(cap_bf16=999), dict(cap_fp8=901)])
def test_one_cache_of_two_shapes(other):
    every = tuple(range(14))
    assert abi.arkv_cache_fork(cfg(), cache(*every), cfg(**other), cache(*every), P, None, check=False) == abi.ARKV_EINVAL
    assert "share no buffer" in abi.arkv_last_error_string()
