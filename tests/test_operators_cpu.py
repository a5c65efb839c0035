"""arkv_qk_norm_rope, arkv_cache_fork, arkv_prefix_attn and arkv_decode_ml refuse bad arguments
before any launch (no CUDA device is touched), and the host-only sizes hold together."""
import ctypes

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


ROPE = dict(cfg=cfg(), n_tok=4, qkv=P, qkv_stride=12 * 64, pos0=P, step=0, length=P, q_weight=P, k_weight=P, eps=1e-6,
            freq=P, rot=64, interleaved=0, n_stride=4, q=P, k=P, v=P, q_obs=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(cfg=cfg(head_dim=96)), dict(n_tok=0), dict(n_stride=3), dict(step=-1), dict(qkv=None), dict(k=None), dict(v=None),
    dict(qkv_stride=12 * 64 - 8), dict(qkv_stride=12 * 64 + 4), dict(rot=66), dict(rot=3), dict(rot=-2),
    dict(freq=None), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")), dict(qkv=P + 8), dict(q=P + 2),
    dict(q_obs=P + 4), dict(freq=P + 4), dict(pos0=P + 2), dict(n_tok=1 << 30, n_stride=1 << 30)])
def test_rope_refusals(bad):
    assert abi.arkv_qk_norm_rope(**{**ROPE, **bad}, check=False) == abi.ARKV_EINVAL
    assert abi.arkv_last_error_string()


@pytest.mark.parametrize("bad", [
    dict(dst_cfg=cfg(hkv=4)), dict(dst_cfg=cfg(head_dim=128)), dict(dst_cfg=cfg(quant_format=1)), dict(dst_cfg=cfg(window=0)),
    dict(src=abi.arkv_layer_cache()), dict(dst=abi.arkv_layer_cache()), dict(src_seq=None), dict(src_seq=P + 2),
    # one cache: the same buffers need the same shapes; some shared buffers are no cache of their own
    dict(src=cache(1), dst_cfg=cfg(batch=2)), dict(src=cache(1), dst_cfg=cfg(cap_fp8=901)), dict(src=cache(0))])
def test_fork_refusals(bad):
    c = dict(dst_cfg=cfg(), dst=cache(1), src_cfg=cfg(), src=cache(100), src_seq=P, stream=None)
    if bad.get("src") is not None and bad["src"].k16 == 0:   # shifted by one: every buffer meets another field's
        bad = dict(src=abi.arkv_layer_cache(*[4096 * (i + (1 if i < 3 else 200)) for i in range(15)]))
    assert abi.arkv_cache_fork(**{**c, **bad}, check=False) == abi.ARKV_EINVAL
    assert abi.arkv_last_error_string()


@pytest.mark.parametrize("bad", [
    dict(cfg=cfg(hq=6, hkv=2)), dict(cfg=cfg(head_dim=128)), dict(cfg=cfg(hkv=4, hq=8)), dict(prefix_cfg=cfg(gamma=-1.0)),
    dict(q=None), dict(o=None), dict(prefix=abi.arkv_layer_cache()), dict(branch_start=None), dict(o_own=None),
    dict(ml_own=None), dict(q=P + 8), dict(o=P + 8), dict(o_own=P + 4), dict(ml=P + 4), dict(ml_own=P + 4),
    dict(branch_start=P + 2), dict(ws=None), dict(ws=P + 16), dict(ws_bytes=-1),
    dict(prefix_cfg=cfg(batch=2000, cap_bf16=1 << 20))])
def test_prefix_refusals(bad):
    c = dict(cfg=cfg(), prefix_cfg=cfg(batch=2), q=P, prefix=cache(), branch_start=P, o_own=P, ml_own=P, o=2 * P, ml=P,
             ws=4 * P, ws_bytes=1 << 34, stream=None)
    c.update(bad)
    if c["ws_bytes"] == -1:
        c["ws_bytes"] = abi.arkv_prefix_workspace_bytes(c["cfg"], c["prefix_cfg"]) - 1
    assert abi.arkv_prefix_attn(**c, check=False) == abi.ARKV_EINVAL
    assert abi.arkv_last_error_string()


def test_prefix_workspace_sizes():
    small = abi.arkv_prefix_workspace_bytes(cfg(batch=1), cfg(batch=1))
    large = abi.arkv_prefix_workspace_bytes(cfg(batch=512), cfg(batch=64))
    assert 0 < small <= large
    assert abi.arkv_prefix_workspace_bytes(cfg(), cfg(head_dim=128)) == 0


def test_decode_ml_is_inside_the_workspace():
    c = cfg()
    need = abi.arkv_workspace_bytes(c, abi.ARKV_WS_DECODE)
    ml = abi.arkv_decode_ml(c, P, need)
    assert P <= ml and ml + 3 * 2 * 4 * 8 <= P + need and ml % 8 == 0
    out = ctypes.c_void_p()
    assert abi.lib().arkv_decode_ml(ctypes.byref(c), P, need - 1, ctypes.byref(out)) == abi.ARKV_EINVAL
    assert abi.lib().arkv_decode_ml(ctypes.byref(c), P, need, None) == abi.ARKV_EINVAL


def test_wrappers_refuse_tensors_of_the_host():
    import torch
    from mixed_precision_kv_arkv_b200 import cache as C
    c = cfg(batch=1, hq=2, hkv=1)
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        C.qk_norm_rope(c, z(1, 256), 1, None, z(1, 1, 1, 64), z(1, 1, 1, 64))
    small = C.LayerCache(cfg(batch=1, cap_bf16=4, cap_fp8=4), "cpu")
    with pytest.raises(ValueError):
        C.fork(small, small, torch.zeros(1, dtype=torch.int32))
