"""Attention over the 8-bit cache where the rows' value scales and their weights lie far apart: the
keys that carry a row's weight keep their precision whatever the scale of a key that weighs
nothing, or that the row does not see.

The bound of a row is that of the attention's other checks: (pr + 2 ds + 2^-18) sum_j w_j |v_j| +
u |O| + half a subnormal step, with pr the rounding of the probabilities (2^-11, in two parts
2^-21) and ds that of the scores, 2^-17 (1 + 2^-4) A with A the largest sum of a score's
magnitudes.  To it comes, for each key, what a probability times its scale loses below the
smallest step of fp16: 2^-38 of the row's largest such product, times a code of at most 448.
"""
import math

import numpy as np
import pytest
import torch

from oracle import rows

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


def cache_of(k, v, fmt):
    """A contiguous cache [B, n, Hkv, d] holding the rows k, v, and the fp64 values of both."""
    B, n, Hkv, d = k.shape
    c = [torch.zeros(k.shape, dtype=torch.uint8, device=DEV).view(FMT[fmt]) for _ in "kv"]
    c += [torch.zeros(B, Hkv, n, device=DEV) for _ in "kv"]
    fa().fa_kvcache_append_quant(*c, k.to(DEV), v.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV))
    (kv, _), (vv, vs) = ((rows.dequantise(*q, fmt), q[1]) for q in (rows.quantise(t, fmt) for t in (k, v)))
    return c, kv, vv, vs.astype(np.float64)


def check(q, c, kv, vv, vs, causal=False, window=(-1, -1), **kw):
    """One KV head; where q is a batch of equal queries, kv and vv may be those of one sequence."""
    Sq, d = q.shape[1], q.shape[3]
    n = kv.shape[1]
    dtype = q.dtype
    out, lse = fa().fa_fwd_kvcache_quant(q.to(DEV), *c, causal=causal, window_size=window, **kw)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    qd = q[:len(kv)].double().numpy()
    x = np.einsum("bihd,bjd->bhij", qd, kv[:, :, 0]) / math.sqrt(d)
    A = np.einsum("bihd,bjd->bhij", np.abs(qd), np.abs(kv[:, :, 0])).max() / math.sqrt(d)
    at, j = np.arange(Sq)[:, None] + n - Sq, np.arange(n)
    ok = np.ones((Sq, n), bool)
    if causal:
        ok &= j <= at
    if window[0] >= 0:
        ok &= j >= at - window[0]
    x = np.where(ok, x, -np.inf)
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    l = p.sum(-1, keepdims=True)
    ref = np.einsum("bhij,bjd->bihd", p / l, vv[:, :, 0])
    size = np.einsum("bhij,bjd->bihd", p / l, np.abs(vv[:, :, 0]))
    least = 2.0 ** -38 * 448 * n * ((p / l) * vs[:, None, None, :, 0]).max(-1)  # [B, H, Sq]
    ds = 2.0 ** -17 * (1 + 2.0 ** -4) * A
    pr = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21
    fi = torch.finfo(dtype)
    bound = (pr + 2 * ds + 2.0 ** -18) * size + fi.eps / 2 * np.abs(ref) + np.transpose(least, (0, 2, 1))[..., None]
    bound += fi.tiny * fi.eps / 2
    err = np.abs(out - ref)
    assert np.all(err <= bound), float((err / bound).max())
    want = (m + np.log(l))[..., 0]
    assert np.all(np.abs(lse - want) <= ds + 2.0 ** -20 * (1 + np.abs(want)))


def rows_of(scores, sizes, d, dtype, heads, Sq=1, seed=0):
    """Queries along one direction, keys along it so that the scores are `scores`, and random values
    whose magnitudes are `sizes`."""
    g = torch.Generator().manual_seed(seed)
    n = len(scores)
    u = torch.sign(torch.randn(d, generator=g))
    q = (u * 2).expand(1, Sq, heads, d).to(dtype)
    k = (u * (scores.double() / (2 * math.sqrt(d)))[:, None])[None, :, None].to(dtype)
    v = torch.randn(1, n, 1, d, generator=g, dtype=torch.float64) * sizes.double()[None, :, None, None]
    return q, k, v.to(dtype)


POWERS = {torch.bfloat16: (0, 40), torch.float16: (-18, 15)}  # of two, of the values
FORMS = [("e4m3", 128), ("int8", 128), ("e4m3", 64), ("int8", 64)]
DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])


@DTYPES
@pytest.mark.parametrize("fmt,d", FORMS)
@pytest.mark.parametrize("heads", [4, 16])
@pytest.mark.parametrize("at", [0, 50, 100])
def test_a_large_row_without_weight(dtype, fmt, d, heads, at):
    """One key of a far larger scale and a weight of 2^-100, before, among and behind the others."""
    lo, hi = POWERS[dtype]
    n = 101
    scores, sizes = torch.zeros(n), torch.full((n,), 2.0 ** lo)
    scores[at], sizes[at] = -100 * math.log(2), 2.0 ** (hi - 3)
    q, k, v = rows_of(scores, sizes, d, dtype, heads, seed=at)
    check(q, *cache_of(k, v, fmt))


@DTYPES
@pytest.mark.parametrize("fmt,d", FORMS)
@pytest.mark.parametrize("Sq,heads", [(2, 4), (4, 4), (5, 5)])
def test_a_large_row_that_some_rows_do_not_see(dtype, fmt, d, Sq, heads):
    """Equal scores; the last key is far larger and only the last query row of each head sees it, and
    the first key is beyond the window of all but the first."""
    lo, hi = POWERS[dtype]
    n = 133
    for big in ((n - 1,), (0,), (0, n - 1)):
        sizes = torch.full((n,), 2.0 ** lo)
        sizes[list(big)] = 2.0 ** (hi - 3)
        q, k, v = rows_of(torch.zeros(n), sizes, d, dtype, heads, Sq, seed=Sq)
        check(q, *cache_of(k, v, fmt), causal=True, window=(n - Sq, -1))


@DTYPES
@pytest.mark.parametrize("fmt,d", FORMS)
def test_scores_rise_as_scales_fall(dtype, fmt, d):
    """Each tile's largest score is a little above the last one's, so that the running max grows by
    less than one (base 2) everywhere, while the scales fall: what the first tiles left must not be
    what the last ones are measured by.  Many sequences on the same blocks, so that one share holds
    a whole one."""
    lo, hi = POWERS[dtype]
    tiles, B = 128, 2400
    step = torch.arange(64 * tiles) // 64
    scores = 0.9 * math.log(2) * (step - (tiles - 1.0))
    low = -35 if dtype == torch.bfloat16 else lo
    sizes = 2.0 ** (low + (hi - 3 - low) * (1 - step.double() / (tiles - 1)))
    q, k, v = rows_of(scores, sizes, d, dtype, 4)
    c, kv, vv, vs = cache_of(k, v, fmt)
    pool = [t[0].unflatten(0, (tiles, 64)) for t in c[:2]]
    pool += [t[0].unflatten(1, (tiles, 64)).transpose(0, 1).contiguous() for t in c[2:]]
    check(q.expand(B, -1, -1, -1).contiguous(), pool, kv, vv, vs,
          block_table=torch.arange(tiles, dtype=torch.int32, device=DEV).expand(B, tiles).contiguous(),
          cache_seqlens=torch.full((B,), 64 * tiles, dtype=torch.int32, device=DEV))


@DTYPES
@pytest.mark.parametrize("fmt,d", FORMS)
def test_rows_without_a_value(dtype, fmt, d):
    """Values of zero (scale 0) where the weight is, and all values zero."""
    lo, hi = POWERS[dtype]
    n = 150
    scores, sizes = torch.zeros(n), torch.full((n,), 2.0 ** lo)
    scores[3:70], sizes[3:70] = 60.0, 0.0
    q, k, v = rows_of(scores, sizes, d, dtype, 4)
    check(q, *cache_of(k, v, fmt))
    check(q, *cache_of(k, torch.zeros_like(v), fmt))
