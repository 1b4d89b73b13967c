"""The q/k norm and rotation, the append into the 8-bit cache and both in one launch at sizes where
a warp takes long stretches of tokens: its slots of the copy ring are filled many times, and the
places and angles of tokens are looked up more than once (32 at a time).  The norm and rotation are
held against the definition in 64 bits on the GPU, the rest bit for bit against the definitions or
the calls that it joins.

Tolerance of the norm and rotation: u |y| + 32 e (|n_a cos| + |n_b sin|) + half a subnormal step, u half
a step of the type, e = 2^-24: a sum of squares of 20 roundings, halved by the root, rsqrt 4, two
products and the rotation's three."""
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


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def table(n, rot):
    ang = torch.arange(n, device=DEV).double()[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, device=DEV).double() / rot)
    return dict(cos=ang.cos().float(), sin=ang.sin().float())


def inputs(shape, H, Hkv, d, dtype, rot, seed):
    """Views q, k, v of one packed projection, weights and tables."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = (randn(g, *shape, H + 2 * Hkv, d) * torch.exp(randn(g, H + 2 * Hkv, 1))).to(dtype)
    kw = dict(q_weight=1 + 0.3 * randn(g, d), k_weight=1 + 0.3 * randn(g, d))
    if rot:
        kw.update(table(41000, rot))
    return qkv[..., :H, :], qkv[..., H:H + Hkv, :], qkv[..., H + Hkv:, :], kw


def check(y, x, w, pos, kw, inter):
    """y [tokens, heads, d] of x, its positions [tokens]."""
    n = x.double()
    n = n / torch.sqrt(n.square().mean(-1, keepdim=True) + 1e-6) * w.double()
    ref, mag = n.clone(), n.abs()
    if "cos" in kw:
        c, s = (kw[t].double()[pos.long()][:, None] for t in ("cos", "sin"))
        rot = 2 * c.shape[-1]

        def parts(t):
            return (t[..., 0:rot:2], t[..., 1:rot:2]) if inter else (t[..., :rot // 2], t[..., rot // 2:rot])

        a, b = (t.clone() for t in parts(n))
        for dst, val in zip(parts(ref), (a * c - b * s, b * c + a * s)):
            dst.copy_(val)
        for dst, val in zip(parts(mag), ((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs())):
            dst.copy_(val)
    err = (y.double() - ref).abs()
    bound = torch.finfo(x.dtype).eps / 2 * ref.abs() + 32 * E * mag + TINY[x.dtype]
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("B,S,H,Hkv,d,dtype,rot,inter", [
    (4, 4096, 32, 8, 128, torch.bfloat16, 128, False),  # 35 steps a warp in one wave: several waves of 12
    (1, 30000, 33, 9, 64, torch.float16, 32, True),
    (2, 9001, 40, 1, 128, torch.float16, 0, False),
    (3000, 7, 17, 20, 64, torch.bfloat16, 64, False),   # 36, many short sequences
])
def test_several_waves(B, S, H, Hkv, d, dtype, rot, inter):
    q, k, _, kw = inputs((B, S), H, Hkv, d, dtype, rot, seed=S)
    g = torch.Generator(device=DEV).manual_seed(1)
    pos = torch.randint(0, 41000, (B, S), generator=g, device=DEV, dtype=torch.int32)
    call = dict(kw, interleaved=inter, positions=pos if rot else None)
    qo, ko = fa().fa_qk_norm_rope(q, k, **call)
    check(qo.flatten(0, 1), q.flatten(0, 1), kw["q_weight"], pos.flatten(), kw, inter)
    check(ko.flatten(0, 1), k.flatten(0, 1), kw["k_weight"], pos.flatten(), kw, inter)
    few = fa().fa_qk_norm_rope(q[-1:, -3:], k[-1:, -3:], **dict(call, positions=pos[-1:, -3:].contiguous() if rot else None))
    assert torch.equal(few[0], qo[-1:, -3:]) and torch.equal(few[1], ko[-1:, -3:])
    q2, k2 = q.contiguous(), k.contiguous()
    got = fa().fa_qk_norm_rope(q2, k2, q_out=q2, k_out=k2, **call)
    assert torch.equal(got[0], qo) and torch.equal(got[1], ko)


def paged(lens, page, Hkv, d, fmt, seed):
    """Pools of zeros with room for lens[b] rows, and their table."""
    need = [-(-n // page) for n in lens]
    n = sum(need) + 2
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).int()
    tab = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(need):
        tab[b, :x] = perm[at:at + x]
        at += x
    t = torch.float8_e4m3fn if fmt == "e4m3" else torch.int8
    pools = [torch.zeros(n, page, Hkv, d, dtype=torch.uint8, device=DEV).view(t) for _ in "kv"]
    return (*pools, *(torch.zeros(n, Hkv, page, device=DEV) for _ in "kv")), tab.to(DEV)


def quantised(x, fmt):
    """Codes (as bytes) and scales of the rows of x."""
    top = 448.0 if fmt == "e4m3" else 127.0
    m = x.double().abs().amax(-1, keepdim=True)
    p = x.double() * top / m
    if fmt == "int8":
        return p.round().to(torch.int8).view(torch.uint8), (m / top).float()[..., 0]
    # the quotient in fp32 lies on the same side of E4M3's rounding borders (2^-19 away, or on them)
    return p.float().to(torch.float8_e4m3fn).view(torch.uint8), (m / top).float()[..., 0]


def places(cu, lens, tab, page, total):
    """Block and row of each packed token."""
    r = torch.arange(total, device=DEV)
    b = torch.searchsorted(cu[1:].long(), r, right=True)
    pos = r - cu.long()[b] + lens.long()[b]
    return tab.long()[b, pos // page], pos % page, pos


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,Hkv,dtype", [(128, 4, torch.bfloat16), (64, 8, torch.float16), (64, 3, torch.bfloat16)])
def test_append_of_many_tokens(fmt, d, Hkv, dtype):
    """One step a token and over 32 tokens a warp; sequences begin and end inside the stretches."""
    new = [60001, 3, 0, 17000, 1, 50, 82950]
    lens = [5, 60, 7, 0, 100, 300, 1000]
    total = sum(new)
    c, tab = paged([a + b for a, b in zip(new, lens)], 64, Hkv, d, fmt, seed=d)
    _, k, v, _ = inputs((total,), 0, Hkv, d, dtype, 0, seed=Hkv)
    cs, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, [0, *torch.tensor(new).cumsum(0).tolist()]))
    want = [t.clone() for t in c]
    fa().fa_kvcache_append_quant(*c, k, v, cs, block_table=tab, cu_seqlens_new=cu)
    blk, row, _ = places(cu, cs, tab, 64, total)
    for i, x in enumerate((k, v)):
        codes, scale = quantised(x, fmt)
        want[i].view(torch.uint8)[blk, row] = codes
        want[2 + i][blk, :, row] = scale
    for a, b in zip(c, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fmt,d,H,Hkv,dtype,rot,inter", [
    ("e4m3", 128, 4, 4, torch.bfloat16, 128, False), ("int8", 64, 8, 8, torch.float16, 32, True),
    ("int8", 128, 3, 1, torch.bfloat16, 64, False)])
def test_step_over_many_tokens(fmt, d, H, Hkv, dtype, rot, inter):
    """The fused step with over 32 tokens a warp, against the definition and the two calls."""
    new, lens = [30001, 2, 9999, 0, 20100], [9, 64, 0, 3, 2000]
    total = sum(new)
    (a, tab), (b, _) = (paged([m + n for m, n in zip(new, lens)], 64, Hkv, d, fmt, seed=H) for _ in "ab")
    q, k, v, kw = inputs((total,), H, Hkv, d, dtype, rot, seed=H)
    cs, cu = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, [0, *torch.tensor(new).cumsum(0).tolist()]))
    call = dict(kw, interleaved=inter)
    qo = fa().fa_qk_norm_rope_append_quant(q, k, v, *a, cs, block_table=tab, cu_seqlens_new=cu, **call)
    _, _, pos = places(cu, cs, tab, 64, total)
    check(qo, q, kw["q_weight"], pos, kw, inter)
    qn, kn = fa().fa_qk_norm_rope(q, k, positions=pos.int(), **call)
    fa().fa_kvcache_append_quant(*b, kn, v, cs, block_table=tab, cu_seqlens_new=cu)
    assert torch.equal(qo, qn)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
