"""The torch helpers refuse tensors whose addresses alone would not say what the caller means --
strided, too short, of another type -- before anything is launched.  No CUDA device is touched: the
tensors are on the host, and each refusal names the tensor (a call whose tensors are all in order
is refused for the device)."""
import pytest
import torch

from mixed_precision_kv_arkv_b200 import abi, build
from mixed_precision_kv_arkv_b200 import cache as C

BF, I32, F32, F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    abi.lib()


def z(*s, dt=BF):
    return torch.zeros(s, dtype=dt)


B, HQ, HKV, D, N, OBS = 3, 4, 2, 64, 5, 7
W = (HQ + 2 * HKV) * D


def rope_args():
    return dict(qkv=z(B * N, W + 8), n_tok=N, freq=z(32, dt=F64), k=z(B, HKV, N, D), v=z(B, HKV, N, D), q=z(B, HQ, N, D),
                q_obs=z(B, HQ, OBS, D), q_weight=z(D), k_weight=z(D), pos0=z(B, dt=I32), length=z(B, dt=I32))


def rope(**bad):
    a = {**rope_args(), **bad}
    c = C.make_cfg(B, HQ, HKV, D, 16, OBS, 1.0, 0.5, 1, 1)
    C.qk_norm_rope(c, a.pop("qkv"), a.pop("n_tok"), a.pop("freq"), a.pop("k"), a.pop("v"), **a)


def test_rope_takes_tensors_in_order():
    for ok in (dict(), dict(qkv=z(B * N, W)), dict(qkv=z(B * N, W + 64)[:, 8:8 + W]), dict(freq=None), dict(q=None, q_obs=None),
               dict(q_weight=None, k_weight=None, pos0=None, length=None), dict(q_weight=z(2 * D)[D:], pos0=z(9, dt=I32)[2:5])):
        with pytest.raises(ValueError, match="CUDA device"):
            rope(**ok)


@pytest.mark.parametrize("name,bad", [
    ("pos0", z(B, 2, dt=I32)[:, 0]), ("pos0", z(B - 1, dt=I32)), ("pos0", z(B + 1, dt=I32)), ("pos0", z(B, dt=torch.int64)),
    ("pos0", z(1, dt=I32).expand(B)),
    ("length", z(B, 2, dt=I32)[:, 1]), ("length", z(1, dt=I32)), ("length", z(B, dt=F32)),
    ("freq", z(64, dt=F64)[::2]), ("freq", z(32, 2, dt=F64)[:, 0]), ("freq", z(32, dt=F32)),
    ("q_weight", z(D // 2)), ("q_weight", z(2 * D)[::2]), ("q_weight", z(D, dt=F32)),
    ("k_weight", z(D - 1)), ("k_weight", z(1).expand(D)),
    ("qkv", z(B * N, W - 8)), ("qkv", z(B * N, W + 64)[:, :W - 64]), ("qkv", z(B * N - 1, W)), ("qkv", z(B * N, 2 * W)[:, ::2]),
    ("qkv", z(B * N * W)),
    ("k", z(B, HKV, N * D)), ("k", z(B, N, HKV, D).transpose(1, 2)), ("v", z(B, HKV, N, D + 64)[..., :D]),
    ("q", z(B, HQ, N + 1, D)), ("q_obs", z(B, HQ, N, D)),
])
def test_rope_refuses(name, bad):
    with pytest.raises(ValueError, match=rf"^{name} must be"):
        rope(**{name: bad})


def branch_args():
    return dict(q=z(B, HQ, D), k_new=z(B, HKV, 1, D), v_new=z(B, HKV, D), ctx_len=z(B, dt=I32), o_own=z(B, HQ, D, dt=F32),
                o=z(B, HQ, D))


def branch(prefix=None, **bad):
    c = C.make_cfg(B, HQ, HKV, D, 4, 4, 1.0, 0.5, 20, 30)
    st = C.new_layer_state(c, 0.5, "cpu")
    if prefix is None:
        prefix = C.new_shared_prefix(c, C.LayerCache(C.make_cfg(1, HQ, HKV, D, 4, 4, 1.0, 0.5, 9, 9), "cpu"))
    C.branch_step(st, prefix, 0, **{**branch_args(), **bad}, reassign_interval=4)


def test_branch_step_takes_tensors_in_order():
    for ok in (dict(), dict(tier_dbg=z(B * HKV, 50, dt=torch.uint8)), dict(q=z(B, HQ, 1, D), o=z(B, HQ * D))):
        with pytest.raises(ValueError, match="CUDA device"):
            branch(**ok)


@pytest.mark.parametrize("name,bad", [
    ("q", z(B, HQ, D // 2)), ("q", z(B - 1, HQ, D)), ("q", z(B, HQ, D, dt=F32)), ("q", z(B, D, HQ).transpose(1, 2)),
    ("k_new", z(B, HQ, D)), ("k_new", z(B, HKV, 2 * D)[..., :D]), ("v_new", z(B, 1, D)), ("v_new", z(B, HKV, 1)),
    ("ctx_len", z(B, 2, dt=I32)[:, 0]), ("ctx_len", z(B - 1, dt=I32)), ("ctx_len", z(B, dt=torch.int64)),
    ("o_own", z(B, HQ, D)), ("o_own", z(B, HKV, D, dt=F32)), ("o", z(B, HKV, D)), ("o", z(1, 1, D).expand(B, HQ, D)),
    ("o", z(B, HQ, D, dt=F32)), ("o", z(B * HQ * D + 4)[4:]), ("tier_dbg", z(B * HKV, 20, dt=torch.uint8)),
    ("tier_dbg", z(B * HKV, 50)), ("o", torch.zeros((B, HQ, D), dtype=BF, device="meta")),
])
def test_branch_step_refuses(name, bad):
    with pytest.raises(ValueError, match=rf"^{name} must be"):
        branch(**{name: bad})


def test_branch_step_refuses_prefixes_of_others():
    mk = lambda batch, hq, dev: C.LayerCache(C.make_cfg(batch, hq, HKV, D, 4, 4, 1.0, 0.5, 9, 9), dev)   # noqa: E731
    need = abi.arkv_prefix_workspace_bytes(C.make_cfg(B, HQ, HKV, D, 4, 4, 1.0, 0.5, 20, 30), mk(1, HQ, "cpu").cfg)
    short = C.SharedPrefix(mk(1, HQ, "cpu"), None, C.Workspace(need - 1, "cpu"))
    other = C.make_cfg(B, 2 * HQ, HKV, D, 4, 4, 1.0, 0.5, 20, 30)
    elsewhere = C.SharedPrefix(mk(1, HQ, "meta"), None, C.Workspace(1 << 24, "cpu"))
    for prefix in (short, C.new_shared_prefix(other, mk(1, 2 * HQ, "cpu")), elsewhere):
        with pytest.raises(ValueError, match="^prefix must be"):
            branch(prefix=prefix)


@pytest.mark.parametrize("prefixes,starts", [(2, None), (2, [0, 2]), (1, [0, 1, 3]), (2, [0, 2, 1]), (3, [0, 2, 1, 3]),
                                             (2, torch.tensor([2, 0, 3]))])
def test_new_shared_prefix_refuses(prefixes, starts):
    c = C.make_cfg(B, HQ, HKV, D, 4, 4, 1.0, 0.5, 20, 30)
    cache = C.LayerCache(C.make_cfg(prefixes, HQ, HKV, D, 4, 4, 1.0, 0.5, 9, 9), "cpu")
    with pytest.raises(ValueError, match="^branch_start must"):
        C.new_shared_prefix(c, cache, starts)


@pytest.mark.parametrize("starts", [[0, 1, 3], (1, 1, 1), torch.tensor([0, 0, 3], dtype=torch.int64), [-4, 2, 90]])
def test_new_shared_prefix_takes(starts):
    c = C.make_cfg(B, HQ, HKV, D, 4, 4, 1.0, 0.5, 20, 30)
    sp = C.new_shared_prefix(c, C.LayerCache(C.make_cfg(2, HQ, HKV, D, 4, 4, 1.0, 0.5, 9, 9), "cpu"), starts)
    assert sp.branch_start.dtype == I32 and sp.branch_start.tolist() == [int(x) for x in starts]
