"""GPU checks of the gradient of the q/k norm and rotation beyond single groups of rows: eps = 0
and heads that do not fill a group, against the definition in 64 bits (on the GPU: the sizes are
large).

Tolerances, with u half a step of the 16-bit type and e = 2^-24:
  dx: u |dx| + 64 e r (|g w| + |n| mean |g w n|) + half a subnormal step: g takes 3 roundings of the
      rotation, r 15 (a sum of squares of 20, halved by the root, and rsqrt), the dot as many again.
  dw: (80 + rows per lane) e sum |g n|: 20 on each product (g and n as above), one per row that a
      lane adds up, then trees over the rows of a group (3), the warps of a block (8), every 32nd
      block (10) and those sums (32).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = 2.0 ** -24
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


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


def inputs(B, S, H, Hkv, d, dtype, rot, seed, max_pos=41000):
    """q and k as views of one packed projection, gradients, weights and the tables' arguments."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    qkv = (randn(B, S, H + 2 * Hkv, d) * torch.exp(randn(H + 2 * Hkv, 1))).to(dtype)
    gq, gk = randn(B, S, H, d).to(dtype), randn(B, S, Hkv, d).to(dtype)
    kw = dict(q_weight=1 + 0.3 * randn(d), k_weight=1 + 0.3 * randn(d))
    if rot:
        ang = torch.arange(max_pos, device=DEV).double()[:, None] * 10000.0 ** (
            -torch.arange(0, rot, 2, device=DEV).double() / rot)
        kw.update(cos=ang.cos().float(), sin=ang.sin().float(),
                  positions=torch.randint(0, max_pos, (B, S), generator=g, device=DEV, dtype=torch.int32))
    return gq, gk, qkv[:, :, :H], qkv[:, :, H:H + Hkv], kw


def turned_back(dy, kw, inter):
    """dy rotated by the opposite angles, and the bound of its terms' magnitudes."""
    if "cos" not in kw:
        return dy, dy.abs()
    c, s = (kw[n].double()[kw["positions"].long()][:, :, None] for n in ("cos", "sin"))
    rot = 2 * c.shape[-1]

    def parts(t):
        return (t[..., 0:rot:2], t[..., 1:rot:2]) if inter else (t[..., :rot // 2], t[..., rot // 2:rot])

    out, mag = dy.clone(), dy.abs()
    a, b = parts(dy)
    (oa, ob), (ma, mb) = parts(out), parts(mag)
    ra, rb = a * c + b * s, b * c - a * s
    na, nb = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    for dst, src in ((oa, ra), (ob, rb), (ma, na), (mb, nb)):
        dst.copy_(src)
    return out, mag


def rows_per_lane(tokens, H, Hkv, d):
    """How many rows a lane adds up at most: the groups of q and k over the warps of two blocks per SM."""
    rpw = 512 // d
    groups = tokens * (-(-H // rpw) - (-Hkv // rpw))
    blocks = min(2 * torch.cuda.get_device_properties(0).multi_processor_count, tokens)
    return -(-groups // max(8 * blocks - 1, 1))


def check(dx, dw, dy, x, w, kw, inter, eps, per):
    dtype = x.dtype
    g, mag = turned_back(dy.double(), kw, inter)
    x, w = x.double(), w.double()
    inv = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    ref = inv * (g * w) - x * inv ** 3 * (x * g * w).mean(-1, keepdim=True)
    n = (x * inv).abs()
    size = inv * (mag * w.abs() + n * (mag * w.abs() * n).mean(-1, keepdim=True))
    err = (dx.double() - ref).abs()
    bound = torch.finfo(dtype).eps / 2 * ref.abs() + 64 * E * size + TINY[dtype]
    assert bool((err <= bound).all()), float((err / bound).max())
    err = (dw.double() - (g * x * inv).sum((0, 1, 2))).abs()
    bound = (80 + per) * E * (mag * n).sum((0, 1, 2))
    assert bool((err <= bound).all()), float((err / bound).max())


def run(B, S, H, Hkv, d, dtype, rot, inter, eps, seed):
    gq, gk, q, k, kw = inputs(B, S, H, Hkv, d, dtype, rot, seed)
    call = dict(kw, interleaved=inter, eps=eps)
    got = fa().fa_qk_norm_rope_bwd(gq, gk, q, k, **call)
    per = rows_per_lane(B * S, H, Hkv, d)
    check(got[0], got[2], gq, q, kw["q_weight"], kw, inter, eps, per)
    check(got[1], got[3], gk, k, kw["k_weight"], kw, inter, eps, per)
    return (gq, gk, q, k, call), got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("d,H,Hkv", [(128, 2, 2), (128, 5, 1), (128, 8, 3), (64, 4, 4), (64, 9, 1), (64, 32, 8)])
def test_no_eps(dtype, d, H, Hkv):
    """eps = 0 with rows that are not zero; the last group of a token's heads is partly empty."""
    run(2, 45, H, Hkv, d, dtype, d // 2, False, 0.0, seed=d + H)


@pytest.mark.parametrize("B,S,H,Hkv,d,dtype,rot,inter", [
    (2, 6001, 32, 8, 128, torch.bfloat16, 128, False),   # 51 groups a warp: a training batch
    (1, 9000, 33, 9, 64, torch.float16, 32, True),       # 27, heads that do not fill a group
    (1, 50001, 4, 4, 128, torch.float16, 64, False),     # one group a token, 43 tokens a warp
    (1, 50001, 3, 8, 64, torch.bfloat16, 64, True),
    (700, 90, 8, 1, 64, torch.bfloat16, 0, False),       # 54, many short sequences, no rotation
])
def test_many_groups_per_warp(B, S, H, Hkv, d, dtype, rot, inter):
    """Each warp's slots of the copy ring are filled many times over, and positions looked up more than
    once; also with the gradients written where the outputs' gradients were."""
    assert rows_per_lane(B * S, H, Hkv, d) >= 8
    (gq, gk, q, k, call), got = run(B, S, H, Hkv, d, dtype, rot, inter, 1e-6, seed=S)
    again = fa().fa_qk_norm_rope_bwd(gq, gk, q, k, **call)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    for _ in range(3):
        a, b = gq.clone(), gk.clone()
        inplace = fa().fa_qk_norm_rope_bwd(a, b, q, k, dq=a, dk=b, **call)
        assert inplace[0] is a and inplace[1] is b
        for x, y in zip(inplace, got):
            assert torch.equal(x, y)
