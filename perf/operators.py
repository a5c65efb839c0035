"""Cases and plain forms of the operators around a shared or forked prompt: the
norm and rotation of queries and keys (arkv_qk_norm_rope), the copying of cached
sequences (arkv_cache_fork) and the attention of many branches to one prefix
(arkv_prefix_attn).

`listed()` and `draw()` give cases (plain dicts), `prepare()` makes what a program
holds before the call, `run()` makes one pass -- in elementary torch operations, or
with `own` set through the library -- `work()` says what a pass cannot do without
and `exact()` what it gives in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
WINDOW = 64   # observation queries of the prefill cases


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of each of 4 sequences, LLaMA3-8B heads: rotation only, where latency counts
        dict(name="rope decode 4", op="rope", hq=32, hkv=8, head_dim=128, batch=4, tokens=1, ragged=False,
             norm=False, rot=128, interleaved=False, start=32768),
        # a serving batch of 96, Qwen3-8B heads: norm and rotation, far positions
        dict(name="norm rope decode 96", op="rope", hq=32, hkv=8, head_dim=128, batch=96, tokens=1, ragged=False,
             norm=True, rot=128, interleaved=False, start=131072),
        # the prompt of one sequence, Qwen3-8B heads, with the last queries kept for the prefill statistics
        dict(name="norm rope prompt 8192", op="rope", hq=32, hkv=8, head_dim=128, batch=1, tokens=8192, ragged=False,
             norm=True, rot=128, interleaved=False, start=0),
        # a padded batch of prompts with small heads, half of each rotated in neighbouring pairs
        dict(name="norm rope ragged prompts", op="rope", hq=8, hkv=2, head_dim=64, batch=5, tokens=1733, ragged=True,
             norm=True, rot=32, interleaved=True, start=0),
        # the small workload's prompt, copied for a second sample
        dict(name="fork tiny 1 to 2", op="fork", hkv=2, head_dim=64, seqs=1, copies=2, kept16=356, kept8=292,
             ragged=False, format="e4m3", in_place=False),
        # a 32K prompt of the LLaMA3-8B shape (a quarter of its bytes kept), forked for 16 samples
        dict(name="fork 32K prompt 1 to 16", op="fork", hkv=8, head_dim=128, seqs=1, copies=16, kept16=5921, kept8=4739,
             ragged=False, format="e4m3", in_place=False),
        # beams of a ragged batch: every fourth sequence replaced by its neighbour's state, in place
        dict(name="reorder 32 ragged", op="fork", hkv=8, head_dim=128, seqs=32, copies=32, kept16=1403, kept8=2811,
             ragged=True, format="e5m2", in_place=True),
        # two samples of a 2048-token prompt, small heads: the smallest call
        dict(name="prefix tiny 2", op="prefix", hq=8, hkv=2, head_dim=64, prefixes=1, branches=2, kept16=356, kept8=292,
             format="e4m3"),
        # four samples of a 32K prompt, LLaMA3-8B heads
        dict(name="prefix 32K 4", op="prefix", hq=32, hkv=8, head_dim=128, prefixes=1, branches=4, kept16=5921,
             kept8=4739, format="e4m3"),
        # 32 requests behind one 32K system prompt
        dict(name="prefix 32K 32", op="prefix", hq=32, hkv=8, head_dim=128, prefixes=1, branches=32, kept16=5921,
             kept8=4739, format="e4m3"),
        # five prompts of different lengths with 23 branches among them, three queries a key head, E5M2
        dict(name="prefix groups 5 of 23", op="prefix", hq=12, hkv=4, head_dim=128, prefixes=5, branches=23,
             kept16=2501, kept8=3999, format="e5m2"),
        # 64 requests behind a 131072-token document, Qwen3-8B heads: the largest
        dict(name="prefix 131K 64", op="prefix", hq=32, hkv=8, head_dim=128, prefixes=1, branches=64, kept16=23701,
             kept8=18900, format="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "fork", "prefix", "prefix"])
    hkv, group, head_dim = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 4), rng.choice([64, 128])
    fmt = rng.choice(["e4m3", "e5m2"])
    if op == "rope":
        decode = rng.random() < 0.5
        return dict(op=op, hq=hkv * group, hkv=hkv, head_dim=head_dim, batch=_log(rng, 1, 200) if decode else rng.randint(1, 4),
                    tokens=1 if decode else _log(rng, WINDOW, 4000), ragged=not decode and rng.random() < 0.5,
                    norm=rng.random() < 0.6, rot=rng.choice([head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)]),
                    interleaved=rng.random() < 0.3, start=_log(rng, 1, 131072) if decode else 0)
    if op == "fork":
        in_place = rng.random() < 0.4
        seqs = rng.randint(2, 24) if in_place else rng.randint(1, 3)
        return dict(op=op, hkv=hkv, head_dim=head_dim, seqs=seqs, copies=seqs if in_place else rng.randint(seqs, 16),
                    kept16=_log(rng, 1, 4000), kept8=_log(rng, 1, 4000), ragged=rng.random() < 0.5, format=fmt,
                    in_place=in_place)
    prefixes = rng.choice([1, 1, 2, rng.randint(3, 9)])
    return dict(op=op, hq=hkv * group, hkv=hkv, head_dim=head_dim, prefixes=prefixes,
                branches=max(prefixes, _log(rng, 1, 64)), kept16=_log(rng, 1, 20000 // prefixes),
                kept8=_log(rng, 1, 20000 // prefixes), format=fmt)


# ------------------------------------------------------------------ sizes that follow from a case
def _counts(case, n):
    """Live bf16 and FP8 slots of each of n sequences: all alike, or (ragged) growing."""
    share = [1.0] * n if not case.get("ragged", True) else [(i + 1) / n for i in range(n)]
    return [[max(1, int(case[key] * s)) for s in share] for key in ("kept16", "kept8")]


def _lengths(case):
    b, n = case["batch"], case["tokens"]
    return [n if not case["ragged"] else max(min(n, WINDOW), n - (n * i) // (2 * b)) for i in range(b)]


def _sources(case):
    """The source of every destination sequence: dealt out evenly, or (in place) every fourth
    sequence takes its neighbour's state and the others stay."""
    if case["in_place"]:
        return [i - 1 if i % 4 == 1 else i for i in range(case["copies"])]
    return [i % case["seqs"] for i in range(case["copies"])]


def _starts(case):
    """First branch of every prefix: the branches dealt out unevenly, one at least each."""
    p, n = case["prefixes"], case["branches"]
    spare, weight = n - p, p * (p + 1) // 2
    return [i + spare * (i * (i + 1) // 2) // weight for i in range(p + 1)]


def _slot_bytes(case):
    d = case["head_dim"]
    return 4 * d + 20, 2 * d + 8 + 20   # K, V, scales, position and score state


def work(case):
    if case["op"] == "rope":
        d, live = case["head_dim"], sum(_lengths(case))
        obs = sum(min(WINDOW, n) for n in _lengths(case)) if case["tokens"] > 1 else 0
        heads = case["hq"] + 2 * case["hkv"]
        return {"bytes": 2 * d * (2 * live * heads + obs * case["hq"]), "flops": 8 * d * live * (case["hq"] + case["hkv"])}
    n16, n8 = _counts(case, case["seqs"] if case["op"] == "fork" else case["prefixes"])
    if case["op"] == "fork":
        b16, b8 = _slot_bytes(case)
        size = [case["hkv"] * (a * b16 + b * b8) for a, b in zip(n16, n8)]
        moved = [s for i, s in enumerate(_sources(case)) if not (case["in_place"] and s == i)]
        return {"bytes": sum(size[s] for s in set(moved)) + sum(size[s] for s in moved), "flops": 0}
    d, hq, hkv, n, st = case["head_dim"], case["hq"], case["hkv"], case["branches"], _starts(case)
    cache = sum(hkv * (a * 4 * d + b * (2 * d + 8)) for a, b in zip(n16, n8))
    pairs = sum((st[i + 1] - st[i]) * hq * (n16[i] + n8[i]) for i in range(case["prefixes"]))
    return {"bytes": cache + n * hq * (2 * d + 4 * d + 2 * d + 16), "flops": 4 * d * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _quantize(x, fmt):
    """FP8 codes and the absmax scale of each vector."""
    s = x.abs().amax(-1) / FMAX[fmt]
    return (x / s[..., None]).to(FP8[fmt]), s


def _fill(cache, g, n16, n8, hkv, fmt, u):
    """Random live slots (a sink, heavy hitters along u) in the segments of a cache."""
    rows, cap16, d = cache["k16"].shape
    cap8 = cache["k8"].shape[1]
    for key, cap in (("16", cap16), ("8", cap8)):
        k, v = _randn(g, rows, cap, d), _randn(g, rows, cap, d)
        ur = u.repeat(rows // hkv, 1)[:, None, :]
        k += 2.0 * ur * (torch.rand((rows, cap, 1), generator=g, device=DEV) < 0.05)
        if key == "16":
            k[:, 0] = 4.0 * ur[:, 0]
            cache["k16"].copy_(k), cache["v16"].copy_(v)
        else:
            for name, x in (("k", k), ("v", v)):
                code, s = _quantize(x, fmt)
                cache[name + "8"].copy_(code.view(torch.uint8))
                cache["s" + name].copy_(s)
        cache["pos" + key].copy_(torch.randperm(cap, generator=g, device=DEV).to(torch.int32).expand(rows, cap))
        tail = "16" if key == "16" else "8"
        cache["mu" + tail].copy_(torch.rand((rows, cap), generator=g, device=DEV).double() * 1e-3)
        cache[("m2_16" if key == "16" else "m2_8")].copy_(torch.rand((rows, cap), generator=g, device=DEV).double() * 1e-5)
    cache["n_bf16"].copy_(torch.tensor(n16, dtype=torch.int32).repeat_interleave(hkv))
    cache["n_fp8"].copy_(torch.tensor(n8, dtype=torch.int32).repeat_interleave(hkv))


FIELDS16 = ("k16", "v16", "pos16", "mu16", "m2_16")
FIELDS8 = ("k8", "v8", "sk", "sv", "pos8", "mu8", "m2_8")


def _buffers(rows, cap16, cap8, d):
    """The buffers of one layer's cache, as the framework's LayerCache holds them."""
    i32, f32, f64, u8, bf = torch.int32, torch.float32, torch.float64, torch.uint8, torch.bfloat16
    z = lambda dt, *s: torch.zeros(s, dtype=dt, device=DEV)   # noqa: E731
    return dict(k16=z(bf, rows, cap16, d), v16=z(bf, rows, cap16, d), pos16=z(i32, rows, cap16), mu16=z(f64, rows, cap16),
                m2_16=z(f64, rows, cap16), k8=z(u8, rows, cap8, d), v8=z(u8, rows, cap8, d), sk=z(f32, rows, cap8),
                sv=z(f32, rows, cap8), pos8=z(i32, rows, cap8), mu8=z(f64, rows, cap8), m2_8=z(f64, rows, cap8),
                n_bf16=z(i32, rows), n_fp8=z(i32, rows), status=z(i32, 1))


def _handle(s, name, case, batch, hq, cap16, cap8):
    """What a program that uses the library holds of a cache: its configuration and addresses."""
    from mixed_precision_kv_arkv_b200 import abi, cache
    c = s[name]
    s[name + "_cfg"] = cache.make_cfg(batch, hq, case["hkv"], case["head_dim"], WINDOW, WINDOW, 1.0, 1.0, cap16, cap8,
                                      case.get("format", "e4m3"))
    s[name + "_c"] = abi.arkv_layer_cache(*[c[n].data_ptr() for n, _ in abi.arkv_layer_cache._fields_])


def prepare(case, seed):
    g = _gen(seed)
    d, hkv, s = case["head_dim"], case["hkv"], {"case": case}
    if case["op"] == "rope":
        b, n, hq = case["batch"], case["tokens"], case["hq"]
        s["qkv"] = _randn(g, b * n, (hq + 2 * hkv) * d).to(torch.bfloat16)
        s["wq"], s["wk"] = [(1.0 + 0.2 * _randn(g, d)).to(torch.bfloat16) for _ in range(2)]
        half = case["rot"] // 2
        s["freq"] = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        s["pos"] = torch.randint(0, max(1, case["start"]), (b,), generator=g, device=DEV, dtype=torch.int32) \
            if case["start"] else torch.zeros(b, dtype=torch.int32, device=DEV)
        s["len"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
        z = lambda h, t: torch.zeros((b, h, t, d), dtype=torch.bfloat16, device=DEV)   # noqa: E731
        s["q"], s["k"], s["v"] = z(hq, n), z(hkv, n), z(hkv, n)
        s["q_obs"] = z(hq, WINDOW) if n > 1 else None
        if own:
            from mixed_precision_kv_arkv_b200 import cache
            s["cfg"] = cache.make_cfg(b, hq, hkv, d, WINDOW, WINDOW, 1.0, 1.0, 1, 1)
        return s
    u = _randn(g, hkv, d)
    u = math.sqrt(d) * u / u.norm(dim=1, keepdim=True)
    seqs = case["seqs"] if case["op"] == "fork" else case["prefixes"]
    n16, n8 = _counts(case, seqs)
    cap16, cap8 = case["kept16"] + 16, case["kept8"] + 16
    s["src"] = _buffers(seqs * hkv, cap16, cap8, d)
    _fill(s["src"], g, n16, n8, hkv, case["format"], u)
    if case["op"] == "fork":
        s["map"] = torch.tensor(_sources(case), dtype=torch.int32, device=DEV)
        s["dst"] = s["src"] if case["in_place"] else _buffers(case["copies"] * hkv, cap16, cap8, d)
        if own:
            _handle(s, "src", case, seqs, hkv, cap16, cap8)
            _handle(s, "dst", case, case["copies"], hkv, cap16, cap8)
        return s
    n, hq = case["branches"], case["hq"]
    q = _randn(g, n, hkv, hq // hkv, d) + 0.5 * u[None, :, None, :]
    s["q"] = q.reshape(n, hq, d).to(torch.bfloat16)
    s["start"] = torch.tensor(_starts(case), dtype=torch.int32, device=DEV)
    s["o_own"] = 0.3 * _randn(g, n, hq, d)
    # each branch's own tokens: the reference of their softmax near the prefix's, and its sum
    ml = torch.zeros((n * hkv, 4, 2), device=DEV)
    ml[..., 0] = 2.0 * d + 12.0 * _randn(g, n * hkv, 4)
    ml[..., 1] = 1.0 + 40.0 * torch.rand((n * hkv, 4), generator=g, device=DEV)
    ml[:, hq // hkv:] = 0.0
    s["ml_own"] = ml
    s["o"] = torch.zeros((n, hq, d), dtype=torch.bfloat16, device=DEV)
    s["ml"] = torch.zeros_like(ml)
    if own:
        from mixed_precision_kv_arkv_b200 import abi, cache
        _handle(s, "src", case, seqs, hq, cap16, cap8)
        s["cfg"] = cache.make_cfg(n, hq, hkv, d, WINDOW, WINDOW, 1.0, 1.0, 1, 1)
        s["ws"] = cache.Workspace(abi.arkv_prefix_workspace_bytes(s["cfg"], s["src_cfg"]), torch.device(DEV))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope_plain, "fork": _fork_plain, "prefix": _prefix_plain}[s["case"]["op"]](s)


def _run_own(s):
    from mixed_precision_kv_arkv_b200 import abi
    from mixed_precision_kv_arkv_b200.cache import stream_ptr
    case, st = s["case"], stream_ptr()
    if case["op"] == "rope":
        norm, many = case["norm"], s["q_obs"] is not None
        abi.arkv_qk_norm_rope(s["cfg"], case["tokens"], s["qkv"].data_ptr(), s["qkv"].shape[1], s["pos"].data_ptr(), 0,
                              s["len"].data_ptr() if case["ragged"] else None, s["wq"].data_ptr() if norm else None,
                              s["wk"].data_ptr() if norm else None, 1e-6, s["freq"].data_ptr(), case["rot"],
                              int(case["interleaved"]), case["tokens"], s["q"].data_ptr(), s["k"].data_ptr(),
                              s["v"].data_ptr(), s["q_obs"].data_ptr() if many else None, st)
        return _rope_out(s)
    if case["op"] == "fork":
        abi.arkv_cache_fork(s["dst_cfg"], s["dst_c"], s["src_cfg"], s["src_c"], s["map"].data_ptr(), st)
        return _fork_out(s)
    abi.arkv_prefix_attn(s["cfg"], s["src_cfg"], s["q"].data_ptr(), s["src_c"], s["start"].data_ptr(),
                         s["o_own"].data_ptr(), s["ml_own"].data_ptr(), s["o"].data_ptr(), s["ml"].data_ptr(),
                         s["ws"].ptr, s["ws"].nbytes, st)
    return {"o": s["o"], "ml": s["ml"]}


def _rope_out(s):
    out = {"q": s["q"], "k": s["k"], "v": s["v"]}
    return out if s["q_obs"] is None else dict(out, q_obs=s["q_obs"])


def _rotate(x, cos, sin, rot, interleaved):
    half = rot // 2
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, rest], -1)


def _rope_plain(s):
    case = s["case"]
    b, n, hq, hkv, d = case["batch"], case["tokens"], case["hq"], case["hkv"], case["head_dim"]
    x = s["qkv"].view(b, n, hq + 2 * hkv, d).transpose(1, 2).float()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if case["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["wq"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["wk"].float()
    t = torch.arange(n, device=DEV)
    angle = (s["pos"].double()[:, None] + t)[:, None, :, None] * s["freq"]   # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = [_rotate(y, cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16) for y in (q, k)]
    live = (t < s["len"][:, None])[:, None, :, None]
    s["q"].copy_(torch.where(live, q, s["q"]))
    s["k"].copy_(torch.where(live, k, s["k"]))
    s["v"].copy_(torch.where(live, v.to(torch.bfloat16), s["v"]))
    if s["q_obs"] is not None:   # the queries of each sequence's last positions
        last = (s["len"][:, None] - WINDOW + torch.arange(WINDOW, device=DEV))[:, None, :, None]
        s["q_obs"].copy_(torch.gather(q, 2, last.long().expand(b, hq, WINDOW, d)))
    return _rope_out(s)


def _fork_out(s):
    dst, t = s["dst"], FP8[s["case"]["format"]]
    return [dst[f].view(t) if f in ("k8", "v8") else dst[f] for f in FIELDS16 + FIELDS8 + ("n_bf16", "n_fp8", "status")]


def _fork_plain(s):
    case, src, dst = s["case"], s["src"], s["dst"]
    hkv = case["hkv"]
    rows = (s["map"].long()[:, None] * hkv + torch.arange(hkv, device=DEV)).flatten()
    n16, n8 = src["n_bf16"][rows], src["n_fp8"][rows]

    def move(f, n):
        x, y = src[f][rows], dst[f]
        live = torch.arange(x.shape[1], device=DEV) < n[:, None]
        y.copy_(torch.where(live[..., None] if x.dim() == 3 else live, x, y))

    [move(f, n16) for f in FIELDS16], [move(f, n8) for f in FIELDS8]
    dst["n_bf16"].copy_(n16), dst["n_fp8"].copy_(n8)
    return _fork_out(s)


def _prefix_plain(s):
    case, c = s["case"], s["src"]
    P, n, hq, hkv, d = case["prefixes"], case["branches"], case["hq"], case["hkv"], case["head_dim"]
    G, fp8 = hq // hkv, FP8[case["format"]]
    k = torch.cat([c["k16"].float(), c["k8"].view(fp8).float() * c["sk"][..., None]], 1)
    v = torch.cat([c["v16"].float(), c["v8"].view(fp8).float() * c["sv"][..., None]], 1)
    live = torch.cat([torch.arange(c["k16"].shape[1], device=DEV) < c["n_bf16"][:, None],
                      torch.arange(c["k8"].shape[1], device=DEV) < c["n_fp8"][:, None]], 1)
    # branches of each prefix side by side: [prefix, key head, branch and query of the group, dim]
    st = _starts(case)
    most = max(b - a for a, b in zip(st, st[1:]))
    at = s["start"][:-1, None].long() + torch.arange(most, device=DEV)
    real = at < s["start"][1:, None]
    at = at.clamp(max=n - 1)
    pack = lambda x: x[at].view(P, most, hkv, G, -1).transpose(1, 2).reshape(P * hkv, most * G, -1)   # noqa: E731
    raw = torch.matmul(pack(s["q"].float()), k.transpose(1, 2))
    raw = torch.where(live[:, None, :], raw, float("-inf"))
    ml = s["ml_own"].view(n, hkv, 4, 2)[:, :, :G].reshape(n, hq, 2)
    m_own, l_own = pack(ml[..., :1].contiguous()), pack(ml[..., 1:].contiguous())
    m = torch.maximum(raw.amax(-1, keepdim=True), m_own)
    p = torch.exp((raw - m) * d ** -0.5)
    w = l_own * torch.exp((m_own - m) * d ** -0.5)
    total = p.sum(-1, keepdim=True) + w
    o = (torch.matmul(p, v) + w * pack(s["o_own"])) / total
    unpack = lambda x: x.view(P, hkv, most, G, -1).transpose(1, 2).reshape(P, most, hkv * G, -1)[real]   # noqa: E731
    s["o"].copy_(unpack(o))
    s["ml"].view(n, hkv, 4, 2)[:, :, :G].copy_(unpack(torch.cat([m, total], -1)).view(n, hkv, G, 2))
    return {"o": s["o"], "ml": s["ml"]}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    was, own = own, False   # the inputs alone: no handle of the library
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rope": _rope_exact, "fork": _fork_exact, "prefix": _prefix_exact}[case["op"]](case, s)


def _rope_exact(case, s):
    b, n, hq, hkv, d, rot = (case[x] for x in ("batch", "tokens", "hq", "hkv", "head_dim", "rot"))
    x = s["qkv"].double().view(b, n, hq + 2 * hkv, d)
    pos = s["pos"].double()[:, None] + torch.arange(n, device=DEV, dtype=torch.float64)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[..., None] * s["freq"])[:, :, None, :]
    out = []
    for lo, hi, w in ((0, hq, s["wq"]), (hq, hq + hkv, s["wk"]), (hq + hkv, hq + 2 * hkv, None)):
        y = x[:, :, lo:hi].clone()
        if w is not None and case["norm"]:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
        if w is not None:
            i = torch.arange(rot // 2, device=DEV)
            ia, ib = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            z = torch.complex(y[..., ia], y[..., ib]) * turn
            y[..., ia], y[..., ib] = z.real, z.imag
        out.append(y.transpose(1, 2).contiguous())
    q_obs = torch.zeros((b, hq, WINDOW, d), dtype=torch.float64, device=DEV)
    for i, length in enumerate(_lengths(case)):
        if n > 1:
            q_obs[i] = out[0][i, :, length - WINDOW:length]
        for y in out:
            y[i, :, length:] = 0.0
    return dict(q=out[0], k=out[1], v=out[2], **({"q_obs": q_obs} if n > 1 else {}))


def _fork_exact(case, s):
    hkv, t = case["hkv"], FP8[case["format"]]
    old, new = s["src"], {f: x.clone() for f, x in s["dst"].items()}
    n16, n8 = _counts(case, case["seqs"])
    for b, a in enumerate(_sources(case)):
        for fields, n in ((FIELDS16, n16[a]), (FIELDS8, n8[a])):
            for f in fields:
                new[f][b * hkv:(b + 1) * hkv, :n] = old[f][a * hkv:(a + 1) * hkv, :n]
    return [new[f].view(t).double() if f in ("k8", "v8") else new[f].double() for f in FIELDS16 + FIELDS8] + [None] * 3


def _prefix_exact(case, s):
    c, hkv, d, fp8 = s["src"], case["hkv"], case["head_dim"], FP8[case["format"]]
    G, st, (n16, n8) = case["hq"] // hkv, _starts(case), _counts(case, case["prefixes"])
    o, ml = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV), s["ml"].double()
    for r in range(case["prefixes"] * hkv):
        pre, g = divmod(r, hkv)
        a, b, br = n16[pre], n8[pre], slice(st[pre], st[pre + 1])
        heads = slice(g * G, (g + 1) * G)
        K, V = [torch.cat([c[x + "16"][r, :a].double(),
                           c[x + "8"][r, :b].view(fp8).double() * c["s" + x][r, :b].double()[:, None]]) for x in "kv"]
        own_row = s["ml_own"].double().view(-1, hkv, 4, 2)[br, g, :G]
        logit = s["q"][br, heads].double() @ K.T
        top = torch.maximum(logit.max(-1).values, own_row[..., 0])
        weight = ((logit - top[..., None]) / math.sqrt(d)).exp()
        w = own_row[..., 1] * ((own_row[..., 0] - top) / math.sqrt(d)).exp()
        total = weight.sum(-1) + w
        o[br, heads] = (weight @ V + w[..., None] * s["o_own"][br, heads].double()) / total[..., None]
        ml.view(-1, hkv, 4, 2)[br, g, :G] = torch.stack([top, total], -1)
    return {"o": o, "ml": ml}
