"""Forms of the attention over the 8-bit cache that the other checks leave out, against plain
attention in 64 bits on the values that the codes stand for (on the GPU).

Bounds, as in the other checks of this operator: with A the largest sum of a score's magnitudes,
ds = 2^-17 (1 + 2^-4) A + softcap 2^-20 + 2^-21 slope distance for the scores;
  LSE: ds + 2^-20 (1 + |LSE|)
  O:   (pr + 2 ds + 2^-18) sum_j w_j |v_j| + u |O| + half a subnormal step, pr the rounding of the
       probabilities (2^-11, for fp16 outputs in two parts 2^-21), u that of the output."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from io_aware_online_b200 import build
    build.build()
    import io_aware_online_b200 as fa
    fa.load()
    fa.fa_device_status(clear=True)
    yield
    assert fa.fa_device_status(clear=True) == 0


def fa():
    import io_aware_online_b200 as m
    return m


def codes(shape, fmt, seed):
    """Random codes over the whole format (an E4M3 NaN left out)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.int16).to(torch.uint8)
    if fmt == "e4m3":
        c = torch.where((c & 0x7f) == 0x7f, c & 0xf7, c)
        return c.view(FMT[fmt])
    return c.view(torch.int8)


def scales(shape, top, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp(0.5 * torch.randn(shape, generator=g, device=DEV)) * (2.0 / top)


def contiguous_cache(B, n, Hkv, d, fmt, heads_first=False, seed=0):
    """k, v codes [B, n, Hkv, d] and scales [B, Hkv, n] of a contiguous cache."""
    shape = (B, Hkv, n, d) if heads_first else (B, n, Hkv, d)
    kv = [codes(shape, fmt, seed + i) for i in range(2)]
    kv = [t.transpose(1, 2) for t in kv] if heads_first else kv
    top = 448.0 if fmt == "e4m3" else 127.0
    return (*kv, *(scales((B, Hkv, n), top, seed + 2 + i) for i in range(2)))


def values(c):
    """fp64 keys and values [B, n, Hkv, d] of a contiguous cache."""
    k, v, ks, vs = c
    return [t.double() * s.double().transpose(1, 2)[..., None] for t, s in ((k, ks), (v, vs))]


def check(out, lse, q, k, v, lens, causal=False, window=(-1, -1), softcap=0.0, slopes=None):
    """Every sequence by itself, every query row and head."""
    B, Sq, H, d = q.shape
    G = H // k.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    pr = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -21
    for b, n in enumerate(lens):
        kb, vb = (t[b, :n].repeat_interleave(G, 1).transpose(0, 1) for t in (k, v))  # [H, n, d]
        qb = q[b].double().transpose(0, 1)
        x = qb @ kb.transpose(1, 2) / math.sqrt(d)
        A = float((qb.abs() @ kb.abs().transpose(1, 2)).max()) / math.sqrt(d) if n else 0.0
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        at = torch.arange(Sq, device=DEV)[:, None] + n - Sq
        j = torch.arange(n, device=DEV)
        far = 0.0
        if slopes is not None:
            x = x - slopes.double()[:, None, None] * (at - j).abs()
            far = float(slopes.max()) * (n + Sq)
        ok = torch.ones(Sq, n, dtype=torch.bool, device=DEV)
        right = 0 if causal else window[1]
        if right >= 0:
            ok &= j <= at + right
        if window[0] >= 0:
            ok &= j >= at - window[0]
        x = x.masked_fill(~ok, -math.inf)
        none = ~ok.any(1)
        rl = torch.logsumexp(x, -1) if n else torch.full((H, Sq), -math.inf, device=DEV, dtype=torch.float64)
        w = torch.exp(x - torch.where(none, 0.0, rl)[..., None])
        ro, size = w @ vb, w @ vb.abs()
        ds = 2.0 ** -17 * (1 + 2.0 ** -4) * A + softcap * 2.0 ** -20 + 2.0 ** -21 * far
        got = lse[b].double()
        assert torch.equal(got == -math.inf, none.expand(H, Sq))
        err = torch.where(none, 0.0, (got - rl).abs())
        assert bool((err <= ds + 2.0 ** -20 * (1 + torch.where(none, 0.0, rl.abs()))).all()), float(err.max())
        err = (out[b].double().transpose(0, 1) - ro).abs()
        bound = (pr + 2 * ds + 2.0 ** -18) * size + u * ro.abs() + 2.0 ** -25
        assert bool((err <= bound).all()), (b, float((err / bound).max()))


def queries(B, Sq, H, d, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(B, Sq, H, d, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 66, 77, 259, 4001])
def test_scales_word_by_word(fmt, d, n):
    """Slabs of an odd number of rows (4001 aside, of a few tiles): the scales do not start on 16
    bytes, so that every lane brings and announces its own.  Many warps begin at once."""
    B = 40 if n < 1000 else 3
    c = contiguous_cache(B, n, 3, d, fmt, seed=n)
    q = queries(B, 2, 6, d, torch.bfloat16, n + 1)
    out, lse = fa().fa_fwd_kvcache_quant(q, *c, causal=True)
    check(out, lse, q, *values(c), [n] * B, causal=True)
    for _ in range(20):
        again = fa().fa_fwd_kvcache_quant(q, *c, causal=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_temporaries_on_another_stream():
    """Arguments that the caller drops right after a call on another stream: their memory is not given
    to the current stream's work while the call still waits to read them."""
    lens = [700, 90]
    c = contiguous_cache(2, 700, 2, 64, "e4m3", True, seed=5)
    q = queries(2, 1, 4, 64, torch.float16, 6)
    cs = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ref = fa().fa_fwd_kvcache_quant(q, *c, cache_seqlens=cs)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        tmp = q.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = fa().fa_fwd_kvcache_quant(tmp, *c, cache_seqlens=cs, stream=stream)
        del tmp
        torch.empty_like(q).fill_(3)  # takes a freed block of that size
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_read_back_rounds_to_fp32_first(fmt, dtype):
    """Bit for bit the product in fp32, rounded to 16 bits; over enough rows that some differ from the
    exact product rounded once."""
    n, Hkv, d = 20000, 4, 64
    c = contiguous_cache(1, n, Hkv, d, fmt, seed=9)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    got = fa().fa_kvcache_read_quant(*c, cu, total=n, dtype=dtype)
    once = 0
    for out, code, scale in zip(got, c[:2], c[2:]):
        s = scale[0].t()[..., None]
        assert torch.equal(out, (code[0].float() * s).to(dtype))
        exact = code[0].double() * s.double()
        err = (out.double() - exact).abs()
        half = torch.finfo(dtype).eps / 2 + 2.0 ** -24
        assert bool((err <= half * exact.abs() + 2.0 ** -25).all())
        # (a double rounds to 16 bits by way of fp32 too, so a wrong rounding shows as an error above half)
        once += int((err > torch.finfo(dtype).eps / 2 * 2.0 ** torch.floor(torch.log2(exact.abs().clamp(min=1e-30)))).sum())
    assert once > 0


LENS = [700, 130, 2048, 5, 1, 0, 333]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Sq,H,Hkv", [(1, 8, 2), (2, 16, 2), (3, 6, 2), (11, 3, 3), (6, 18, 3)])
@pytest.mark.parametrize("terms", ["none", "softcap", "alibi", "both"])
def test_every_variant(fmt, d, dtype, Sq, H, Hkv, terms):
    """Both formats, head dims and types, up to 8, 16 and 36 query rows per KV head, with and without the
    terms that need code of their own."""
    c = contiguous_cache(len(LENS), 2048, Hkv, d, fmt, d == 64, seed=Sq + d)
    q = queries(len(LENS), Sq, H, d, dtype, H)
    kw = dict(causal=Sq != 3)
    if terms in ("softcap", "both"):
        kw["softcap"] = 12.0
    slopes = 2.0 ** -torch.arange(1, H + 1, device=DEV).float() if terms in ("alibi", "both") else None
    if terms == "both":
        kw["window"] = (500, 2)
    call = {("window_size" if k == "window" else k): v for k, v in kw.items()}
    cs = torch.tensor(LENS, dtype=torch.int32, device=DEV)
    out, lse = fa().fa_fwd_kvcache_quant(q, *c, cache_seqlens=cs, alibi_slopes=slopes, **call)
    check(out, lse, q, *values(c), LENS, slopes=slopes, **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("Sq,H,Hkv", [(1, 8, 8), (2, 16, 2), (5, 8, 2)])
def test_long_shares(fmt, d, dtype, Sq, H, Hkv):
    """Many tiles a warp, so that its buffers are refilled often, and shares that end inside most pairs."""
    lens = [9000, 20001, 64, 15000, 7777, 1, 12000]
    c = contiguous_cache(len(lens), 20001 + 3, Hkv, d, fmt, True, seed=d)
    q = queries(len(lens), Sq, H, d, dtype, 3)
    cs = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = fa().fa_fwd_kvcache_quant(q, *c, cache_seqlens=cs, causal=True)
    check(out, lse, q, *values(c), lens, causal=True)
    for _ in range(5):
        again = fa().fa_fwd_kvcache_quant(q, *c, cache_seqlens=cs, causal=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
