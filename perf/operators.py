"""The operators around the attention calls, as cases that can be timed and compared.

Five passes, as a program calls them:
  norm_rope       RMS norm of every query and key head and the position rotation
  norm_rope_grad  its gradient with respect to q, k and the two norm weights
  cache           new keys and values quantised into an 8-bit cache, then the sequences
                  read back from it in 16 bits (what a chunked prefill attends)
  attend          a few new query rows per sequence against the 8-bit cache
  step            the input side of a serving step: norm, rotation, the keys and values
                  quantised into the cache, and the new rows read back

With `own` false, run() computes plain forms in elementary torch operations; with `own`
true it makes the calls of io_aware_online_b200.  exact() computes the definitions in
64 bits.

Definitions.  Norm: x * rsqrt(mean(x^2) + eps) * w over the head dim.  Rotation of the
first `rot` elements: (a, b) -> (a cos - b sin, b cos + a sin), a and b half of `rot`
apart or adjacent (interleaved).  Cache: per (token, KV head) row with largest magnitude
m, the scale is m / top, a code is round(x * top / m), top = 127 (int8, ties to even) or
448 (E4M3); a row stands for code * scale.  Attention:
softmax(mask(softcap(scale q k) + ALiBi)) v and the natural-log sum of exponentials, masks
aligned to the last key.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
TOP = {"e4m3": 448.0, "int8": 127.0}
EPS = 1e-6
MAX_POS = 40960  # rows of the cos and sin tables


def listed():
    train = {"H": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "rot": 128, "interleaved": False}
    return [
        # a training or prefill batch before its attention forward
        {"name": "norm_rope prefill 4x4096", "op": "norm_rope", "B": 4, "S": 4096, **train},
        # one decoding step of 64 sequences, partial rotation in adjacent pairs: latency
        {"name": "norm_rope decode 64x1", "op": "norm_rope", "B": 64, "S": 1, "H": 32, "Hkv": 8,
         "d": 64, "dtype": "fp16", "rot": 32, "interleaved": True},
        # the backward pass of a training step, an odd length
        {"name": "norm_rope_grad 2x6001", "op": "norm_rope_grad", "B": 2, "S": 6001, **train},
        # the backward pass of a small packed batch
        {"name": "norm_rope_grad 1x333", "op": "norm_rope_grad", "B": 1, "S": 333, "H": 16,
         "Hkv": 4, "d": 64, "dtype": "fp16", "rot": 64, "interleaved": True},
        # a long prompt written into an empty paged cache and read back
        {"name": "cache prompt 4x8192 e4m3", "op": "cache", "B": 4, "lo": 0, "hi": 0, "new_lo": 8192,
         "new_hi": 8192, "Hkv": 8, "d": 128, "dtype": "bf16", "fmt": "e4m3", "page": 256},
        # ragged prompts behind ragged prefixes, small pages
        {"name": "cache ragged 16 int8", "op": "cache", "B": 16, "lo": 3, "hi": 700, "new_lo": 256,
         "new_hi": 8192, "Hkv": 8, "d": 64, "dtype": "fp16", "fmt": "int8", "page": 64},
        # single new tokens behind short prefixes: latency
        {"name": "cache decode 64x1 int8", "op": "cache", "B": 64, "lo": 16, "hi": 200, "new_lo": 1,
         "new_hi": 1, "Hkv": 8, "d": 128, "dtype": "bf16", "fmt": "int8", "page": 64},
        # a full serving batch: single tokens against long ragged paged caches
        {"name": "attend 64x1 to 32768 e4m3", "op": "attend", "B": 64, "Sq": 1, "lo": 1024,
         "hi": 32768, "H": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "fmt": "e4m3", "page": 256,
         "causal": False, "window": -1, "softcap": 0.0, "alibi": False},
        # one long sequence, a contiguous cache, no shared heads: the split over the keys
        {"name": "attend 1x1 to 32749 int8", "op": "attend", "B": 1, "Sq": 1, "lo": 32749,
         "hi": 32749, "H": 16, "Hkv": 16, "d": 64, "dtype": "fp16", "fmt": "int8", "page": 0,
         "causal": False, "window": -1, "softcap": 0.0, "alibi": False},
        # three drafted tokens per sequence, every mask and score term
        {"name": "attend 13x3 masked int8", "op": "attend", "B": 13, "Sq": 3, "lo": 100, "hi": 9000,
         "H": 16, "Hkv": 4, "d": 128, "dtype": "bf16", "fmt": "int8", "page": 64, "causal": True,
         "window": 4096, "softcap": 30.0, "alibi": True},
        # the input side of a decoding step
        {"name": "step 64x1 e4m3", "op": "step", "B": 64, "lo": 1024, "hi": 32768, "new_lo": 1,
         "new_hi": 1, "H": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "rot": 128,
         "interleaved": False, "fmt": "e4m3", "page": 256},
        # the input side of a chunked prefill, ragged chunks
        {"name": "step chunks 4x2048 int8", "op": "step", "B": 4, "lo": 4000, "hi": 6144,
         "new_lo": 1500, "new_hi": 2048, "H": 32, "Hkv": 8, "d": 64, "dtype": "fp16", "rot": 64,
         "interleaved": False, "fmt": "int8", "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "cache", "attend", "attend", "step"])
    Hkv, G = rng.choice([(1, 8), (2, 8), (4, 4), (8, 4), (8, 1), (8, 2), (6, 3), (5, 1), (3, 5)])
    d = rng.choice([64, 128])
    c = {"op": op, "Hkv": Hkv, "d": d, "dtype": rng.choice(["bf16", "fp16"])}
    if op != "cache":
        c["H"] = Hkv * G
    if op in ("norm_rope", "norm_rope_grad", "step"):
        c["rot"] = rng.choice([d, d, d // 2, 16])
        c["interleaved"] = rng.random() < 0.4
    if op in ("cache", "attend", "step"):
        c["fmt"] = rng.choice(["e4m3", "int8"])
        c["page"] = rng.choice([0, 64, 128, 256])
    if op in ("norm_rope", "norm_rope_grad"):
        c["S"] = _log(rng, 1, 8192)
        c["B"] = max(1, min(_log(rng, 1, 64), 12000 // c["S"]))
    elif op == "attend":
        c["Sq"] = rng.choice([1, 1, 1, 2, 3, 4])
        c["hi"] = _log(rng, 40, 30000)
        c["B"] = max(1, min(_log(rng, 1, 64), 900000 // c["hi"]))
        c["lo"] = rng.choice([1, max(1, c["hi"] // 4), c["hi"]])
        c["causal"] = rng.random() < 0.6
        c["window"] = rng.choice([-1, -1, _log(rng, 16, 8000)])
        c["softcap"] = rng.choice([0.0, 0.0, 20.0])
        c["alibi"] = rng.random() < 0.25
    else:
        c["new_hi"] = _log(rng, 1, 8000)
        c["new_lo"] = rng.choice([1, c["new_hi"]])
        c["hi"] = _log(rng, 1, 2900)
        c["B"] = max(1, min(_log(rng, 1, 64), 40000 // (c["new_hi"] + c["hi"])))
        c["lo"] = rng.choice([0, c["hi"]])
    return c


# ------------------------------------------------------------------ inputs
def _lengths(lo, hi, n, seed):
    """n whole numbers in lo .. hi, from the seed, on the host."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _qkv(rows, heads, kv_heads, d, dtype, g):
    """The output of one projection and its q, k, v views; heads differ in size, as they do."""
    qkv = _randn((*rows, heads + 2 * kv_heads, d), torch.float32, g)
    qkv *= torch.exp(_randn((heads + 2 * kv_heads, 1), torch.float32, g) * 0.7)
    qkv = qkv.to(dtype)
    return qkv[..., :heads, :], qkv[..., heads:heads + kv_heads, :], qkv[..., heads + kv_heads:, :]


def _tables(rot):
    """cos and sin of position * 10000^(-2 i / rot), i < rot / 2."""
    pos = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = pos[:, None] * inv
    return a.cos().float(), a.sin().float()


def _norm_inputs(case, g):
    d = case["d"]
    cos, sin = _tables(case["rot"])
    return {"wq": 1 + 0.2 * _randn((d,), torch.float32, g), "wk": 1 + 0.2 * _randn((d,), torch.float32, g),
            "cos": cos, "sin": sin, "interleaved": case["interleaved"]}


def _cache(case, lens, capacity, g, seed):
    """Caches that hold lens[b] quantised rows per sequence (and stale rows behind them) with room
    for capacity[b] rows: pools and a block table in random order, or one slab per sequence."""
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    s = {}
    if page:
        need = (capacity + page - 1) // page
        n = int(need.sum()) + 3
        order = torch.randperm(n, generator=torch.Generator().manual_seed(seed + 7))
        table = torch.full((B, max(1, int(need.max()))), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + int(need[b])].int()
            at += int(need[b])
        s["table"] = table.cuda()
        shape, scales = (n, page, Hkv, d), (n, Hkv, page)
    else:
        s["table"] = None
        rows = int(capacity.max())
        shape, scales = (B, rows, Hkv, d), (B, Hkv, rows)
    top = TOP[case["fmt"]]
    for name in ("k", "v"):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn if case["fmt"] == "e4m3" else torch.int8, device="cuda")
        flat = codes.view(-1, d)
        for i in range(0, flat.shape[0], 1 << 19):
            x = torch.randn((min(1 << 19, flat.shape[0] - i), d), generator=g, device="cuda")
            x = x * (top / x.abs().amax(1, keepdim=True))
            flat[i:i + (1 << 19)] = x.to(codes.dtype) if case["fmt"] == "e4m3" else x.round().to(torch.int8)
        s[name + "_cache"] = codes
        s[name + "_scale"] = torch.exp(0.3 * torch.randn(scales, generator=g, device="cuda")) * (3.0 / top)
    s["lens"] = lens.int().cuda()
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    d = case["d"]
    s = {"case": dict(case), "dtype": dt}
    if op in ("norm_rope", "norm_rope_grad"):
        B, S = case["B"], case["S"]
        s["q"], s["k"], _ = _qkv((B, S), case["H"], case["Hkv"], d, dt, g)
        start = _lengths(0, MAX_POS - S, B, seed).cuda()
        s["positions"] = (start[:, None] + torch.arange(S, device="cuda")).int()
        s.update(_norm_inputs(case, g))
        if op == "norm_rope_grad":
            s["gq"] = _randn((B, S, case["H"], d), dt, g)
            s["gk"] = _randn((B, S, case["Hkv"], d), dt, g)
        return s
    if op == "attend":
        lens = _lengths(case["lo"], case["hi"], case["B"], seed)
        s.update(_cache(case, lens, lens, g, seed))
        s["q"] = _randn((case["B"], case["Sq"], case["H"], d), dt, g)
        s["slopes"] = None
        if case["alibi"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["H"] + 1, device="cuda") / case["H"]).float()
        return s
    # the lengths are the case's own: outputs of one case have one shape
    lens = _lengths(case["lo"], case["hi"], case["B"], 1000 + case["hi"])
    new = _lengths(case["new_lo"], case["new_hi"], case["B"], 2000 + case["new_hi"])
    s.update(_cache(case, lens, lens + new, g, seed))
    s["cu_new"] = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)]).int().cuda()
    total = int(new.sum())
    q, s["k"], s["v"] = _qkv((total,), case.get("H", 0), case["Hkv"], d, dt, g)
    if op == "step":
        s["q"] = q
        s["rows"] = total
        s.update(_norm_inputs(case, g))
    else:
        s["cu_all"] = torch.cat([torch.zeros(1, dtype=torch.long), (lens + new).cumsum(0)]).int().cuda()
        s["rows"] = int((lens + new).sum())
    return s


# ------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, inter, back=False):
    """Rotates x [..., heads, d] by the rows cos, sin [..., rot / 2] (back: by the opposite angle)."""
    cos, sin = cos[..., None, :], sin[..., None, :]
    if back:
        sin = -sin
    rot = 2 * cos.shape[-1]
    t = x[..., :rot]
    a, b = (t[..., 0::2], t[..., 1::2]) if inter else (t[..., :rot // 2], t[..., rot // 2:])
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if inter else -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_norm_rope(x, w, cos, sin, inter):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    return _turn(y, cos, sin, inter).to(x.dtype)


def _plain_norm_rope_grad(gy, x, w, cos, sin, inter):
    gn = _turn(gy.float(), cos, sin, inter, back=True)
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    n = x32 * r
    dw = (gn * n).flatten(0, -2).double().sum(0).float()
    gn = gn * w
    return ((gn - n * (gn * n).mean(-1, keepdim=True)) * r).to(x.dtype), dw


def _quantise(x, fmt):
    """Codes and scales of the rows of x; the quotient in 64 bits, so that no border moves."""
    top = TOP[fmt]
    m = x.float().abs().amax(-1, keepdim=True)
    p = x.double() * top / torch.where(m > 0, m, 1.0).double()
    codes = p.float().to(torch.float8_e4m3fn) if fmt == "e4m3" else p.round().to(torch.int8)
    return codes, (m / top).squeeze(-1)


def _slots(s, cu, start, rows):
    """Block (or sequence) and row within it of packed rows 0 .. rows-1, whose sequence b begins at start[b]."""
    r = torch.arange(rows, device="cuda")
    b = torch.searchsorted(cu[1:].long(), r, right=True)
    pos = r - cu.long()[b] + (0 if start is None else start.long()[b])
    if s["table"] is None:
        return b, pos
    page = s["k_cache"].shape[1]
    return s["table"].long()[b, pos // page], pos % page


def _plain_append(s, k, v):
    blk, row = _slots(s, s["cu_new"], s["lens"], k.shape[0])
    for name, x in (("k", k), ("v", v)):
        codes, scale = _quantise(x, s["case"]["fmt"])
        s[name + "_cache"].view(torch.uint8)[blk, row] = codes.view(torch.uint8)
        s[name + "_scale"][blk, :, row] = scale


def _plain_read(s, cu, start):
    blk, row = _slots(s, cu, start, s["rows"])
    out = []
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        codes = cache.view(torch.uint8)[blk, row].view(cache.dtype).float()
        out.append((codes * s[name + "_scale"][blk, :, row][..., None]).to(s["dtype"]))
    return out


def _allowed(case, lens, keys):
    """[B, Sq, keys]: which keys each query row sees."""
    j = torch.arange(keys, device="cuda")
    at = lens.long()[:, None] - case["Sq"] + torch.arange(case["Sq"], device="cuda")
    ok = (j < lens.long()[:, None, None]).expand(-1, case["Sq"], -1)
    if case["causal"]:
        ok = ok & (j <= at[..., None])
    if case["window"] >= 0:
        ok = ok & (j >= at[..., None] - case["window"])
    return ok, (at[..., None] - j).abs()


def _plain_attend(s):
    case, q = s["case"], s["q"]
    B, Sq, H, d = q.shape
    Hkv = case["Hkv"]

    def values(name):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        if s["table"] is not None:
            t = s["table"].long().clamp(min=0)
            x = cache.view(torch.uint8)[t].view(cache.dtype).float()
            x *= scale[t].transpose(2, 3)[..., None]
            return x.flatten(1, 2)
        return cache.float() * scale.transpose(1, 2)[..., None]

    k = values("k")
    qg = q.float().view(B, Sq, Hkv, H // Hkv, d)
    x = torch.einsum("bihgd,bjhd->bhgij", qg, k) / math.sqrt(d)
    ok, far = _allowed(case, s["lens"], k.shape[1])
    del k
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    if s["slopes"] is not None:
        x = x - s["slopes"].view(Hkv, -1, 1, 1) * far[:, None, None]
    x = x.masked_fill(~ok[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    del x
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1).flatten(1, 2)
    v = values("v")
    v = v.masked_fill(~ok.any(1)[..., None, None], 0.0)
    o = torch.einsum("bhgij,bjhd->bhgid", p, v) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, H, d).to(q.dtype), lse


def _step_positions(s):
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["cu_new"][1:].long(), r, right=True)
    return r - s["cu_new"].long()[b] + s["lens"].long()[b]


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_rope":
        cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
        return (_plain_norm_rope(s["q"], s["wq"], cos, sin, s["interleaved"]),
                _plain_norm_rope(s["k"], s["wk"], cos, sin, s["interleaved"]))
    if op == "norm_rope_grad":
        cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
        dq, dwq = _plain_norm_rope_grad(s["gq"], s["q"], s["wq"], cos, sin, s["interleaved"])
        dk, dwk = _plain_norm_rope_grad(s["gk"], s["k"], s["wk"], cos, sin, s["interleaved"])
        return dq, dk, dwq, dwk
    if op == "cache":
        _plain_append(s, s["k"], s["v"])
        return (*_plain_read(s, s["cu_all"], None), s["k_scale"], s["v_scale"])
    if op == "attend":
        return _plain_attend(s)
    pos = _step_positions(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _plain_norm_rope(s["q"], s["wq"], cos, sin, s["interleaved"])
    k = _plain_norm_rope(s["k"], s["wk"], cos, sin, s["interleaved"])
    _plain_append(s, k, s["v"])
    return (q, *_plain_read(s, s["cu_new"], s["lens"]))


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import io_aware_online_b200 as fa
    op = s["case"]["op"]
    if op == "norm_rope":
        return fa.fa_qk_norm_rope(s["q"], s["k"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                  cos=s["cos"], sin=s["sin"], positions=s["positions"],
                                  interleaved=s["interleaved"])
    if op == "norm_rope_grad":
        return fa.fa_qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], q_weight=s["wq"],
                                      k_weight=s["wk"], eps=EPS, cos=s["cos"], sin=s["sin"],
                                      positions=s["positions"], interleaved=s["interleaved"])
    caches = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "cache":
        fa.fa_kvcache_append_quant(*caches, s["k"], s["v"], s["lens"], block_table=s["table"],
                                   cu_seqlens_new=s["cu_new"])
        k, v = fa.fa_kvcache_read_quant(*caches, s["cu_all"], total=s["rows"], dtype=s["dtype"],
                                        block_table=s["table"])
        return k, v, s["k_scale"], s["v_scale"]
    if op == "attend":
        c = s["case"]
        return fa.fa_fwd_kvcache_quant(s["q"], *caches, cache_seqlens=s["lens"],
                                       block_table=s["table"], causal=c["causal"],
                                       window_size=(c["window"], -1), softcap=c["softcap"],
                                       alibi_slopes=s["slopes"])
    q = fa.fa_qk_norm_rope_append_quant(s["q"], s["k"], s["v"], *caches, s["lens"],
                                        q_weight=s["wq"], k_weight=s["wk"], eps=EPS, cos=s["cos"],
                                        sin=s["sin"], interleaved=s["interleaved"],
                                        block_table=s["table"], cu_seqlens_new=s["cu_new"])
    k, v = fa.fa_kvcache_read_quant(*caches, s["cu_new"], total=s["rows"], dtype=s["dtype"],
                                    seq_start=s["lens"], block_table=s["table"])
    return q, k, v


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ floors
def work(case):
    op, d = case["op"], case["d"]
    H, Hkv = case.get("H", 0), case["Hkv"]
    if op in ("norm_rope", "norm_rope_grad"):
        rows = case["B"] * case["S"]
        x = rows * (H + Hkv) * d
        table = rows * (4 * case["rot"] + 4)
        if op == "norm_rope":
            return {"bytes": 4 * x + table + 8 * d, "flops": 8 * x}
        return {"bytes": 6 * x + table + 16 * d, "flops": 18 * x}
    mean = (case["lo"] + case["hi"]) / 2
    if op == "attend":
        keys = case["hi"] if case["lo"] == case["hi"] else mean
        if case["window"] >= 0:
            keys = min(keys, case["window"] + case["Sq"])
        cached = case["B"] * Hkv * keys
        rows = case["B"] * case["Sq"] * H
        return {"bytes": int(cached * 2 * (d + 4) + rows * (4 * d + 4) + 4 * case["B"]),
                "flops": int(4 * cached * (H // Hkv) * case["Sq"] * d)}
    new = case["B"] * (case["new_lo"] + case["new_hi"]) / 2
    row = Hkv * (d + 4) * 2  # one token's codes and scales, K and V
    wide = Hkv * d * 2 * 2  # the same in 16 bits
    if op == "cache":
        whole = new + case["B"] * mean
        return {"bytes": int(new * (wide + row) + whole * (row + wide)), "flops": int((new + whole) * Hkv * d * 4)}
    return {"bytes": int(new * (wide + row + row + wide + 4 * H * d + 4 * case["rot"])),
            "flops": int(new * (8 * (H + Hkv) * d + 8 * Hkv * d))}


# ------------------------------------------------------------------ 64 bits
def _exact_turn(x, s, pos, sign):
    """x [rows, heads, d] in 64 bits, each row rotated by its position's angle times sign."""
    y = x.clone()
    half = s["cos"].shape[1]
    c, n = s["cos"].double()[pos][:, None], sign * s["sin"].double()[pos][:, None]
    i = torch.arange(half, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    y[..., ia] = x[..., ia] * c - x[..., ib] * n
    y[..., ib] = x[..., ib] * c + x[..., ia] * n
    return y


def _exact_norm(x, w, s, pos):
    x = x.double()
    return _exact_turn(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double(), s, pos, 1.0)


def _exact_grad(gy, x, w, s, pos):
    g = _exact_turn(gy.double(), s, pos, -1.0)
    x = x.double()
    d = x.shape[-1]
    inv = 1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    gw = g * w.double()
    dx = inv * gw - inv ** 3 * x * (gw * x).sum(-1, keepdim=True) / d
    return dx, (g * x * inv).sum((0, 1))


def _exact_rows(x, fmt):
    """What the quantised rows of x stand for, and their scales."""
    x, top = x.double(), TOP[fmt]
    m = x.abs().amax(-1, keepdim=True)
    p = torch.where(m > 0, x * top / m, 0.0)
    if fmt == "int8":
        c = p.round()
    else:  # 3 stored bits of mantissa, exponents from -6, steps of 2^-9 below them
        _, e = torch.frexp(p)
        step = torch.exp2((e - 4).clamp(min=-9).double())
        c = (p / step).round() * step
    return c * (m / top), (m / top).squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op in ("norm_rope", "norm_rope_grad"):
        pos = s["positions"].flatten().long()
        out = []
        for name, w in (("q", s["wq"]), ("k", s["wk"])):
            x = s[name].flatten(0, 1)
            if op == "norm_rope":
                out.append(_exact_norm(x, w, s, pos).view(s[name].shape))
            else:
                out.append(_exact_grad(s["g" + name].flatten(0, 1), x, w, s, pos))
        if op == "norm_rope":
            return out[0], out[1]
        return out[0][0].view(s["q"].shape), out[1][0].view(s["k"].shape), out[0][1], out[1][1]
    if op == "attend":
        return _exact_attend(s)
    lens, cu = s["lens"].tolist(), s["cu_new"].tolist()
    page = case["page"]
    keys = s["k"]
    if op == "step":
        at = torch.cat([torch.arange(n, n + cu[b + 1] - cu[b], device="cuda") for b, n in enumerate(lens)])
        q = _exact_norm(s["q"], s["wq"], s, at)
        keys = _exact_norm(s["k"], s["wk"], s, at).to(s["dtype"])
    rows = {"k": _exact_rows(keys, case["fmt"]), "v": _exact_rows(s["v"], case["fmt"])}
    if op == "step":
        return q, rows["k"][0], rows["v"][0]
    out, scales = [], []
    for name in ("k", "v"):
        scale = s[name + "_scale"].double()
        parts = []
        for b, n in enumerate(lens):
            vals, sc = (t[cu[b]:cu[b + 1]] for t in rows[name])
            whole = n + cu[b + 1] - cu[b]
            for x in range(0, whole, page or max(1, whole)):
                blk = int(s["table"][b, x // page]) if page else b
                r = min(page or whole, whole - x)  # rows of this block that the sequence uses
                kept = max(0, min(r, n - x))       # rows that were there before
                old = s[name + "_cache"][blk, :kept].double() * scale[blk, :, :kept].t()[..., None]
                first = max(0, x - n)
                fresh = slice(first, first + r - kept)
                scale[blk, :, kept:r] = sc[fresh].t()
                parts += [old, vals[fresh]]
        out.append(torch.cat(parts))
        scales.append(scale)
    return (*out, *scales)


def _exact_attend(s):
    case, q = s["case"], s["q"].double()
    B, Sq, H, d = q.shape
    G, page = H // case["Hkv"], case["page"]
    o = torch.zeros_like(q)
    lse = torch.full((B, H, Sq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        kv = []
        for name in ("k", "v"):
            if page:
                blocks = s["table"][b, :(n + page - 1) // page].long()
                codes = s[name + "_cache"].view(torch.uint8)[blocks].view(s["k_cache"].dtype)
                x = codes.double() * s[name + "_scale"][blocks].double().transpose(1, 2)[..., None]
                kv.append(x.flatten(0, 1)[:n])
            else:
                kv.append(s[name + "_cache"][b, :n].double() * s[name + "_scale"][b, :, :n].double().t()[..., None])
        j = torch.arange(n, device="cuda")
        for i in range(Sq):
            at = n - Sq + i
            see = torch.ones(n, dtype=torch.bool, device="cuda")
            if case["causal"]:
                see &= j <= at
            if case["window"] >= 0:
                see &= j >= at - case["window"]
            if not bool(see.any()):
                continue
            x = torch.einsum("hgd,jhd->hgj", q[b, i].view(-1, G, d), kv[0][see]).flatten(0, 1) / math.sqrt(d)
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if s["slopes"] is not None:
                x = x - s["slopes"].double()[:, None] * (j[see] - at).abs()
            lse[b, :, i] = torch.logsumexp(x, 1)
            w = torch.softmax(x, 1).view(-1, G, x.shape[1])
            o[b, i] = torch.einsum("hgj,jhd->hgd", w, kv[1][see]).flatten(0, 1)
    return o, lse
