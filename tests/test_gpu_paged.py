"""Paged caches on the GPU: cache_write, cache_read, paged_forward and paged_decode against
their definitions in 64 bits (tests/paged_ref.py), at the sizes, masks and orders where they
can go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402
from attention_forward_sm_gb300 import binding as attn  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, E4M3 = ref.BF16, ref.E4M3
PAGES = [16, 32, 64, 128]


def _randn(shape, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(BF16).cuda()


def check_attention(o, lse, q, cache, offsets, causal=True, scale=None, more=0.0):
    """|dO| <= 2^-8 (sum_j w_j |v_j| + |O|): a weight and the output are each rounded to bf16
    once, off by half a step, 2^-8, at most; a fiftieth more for everything in 32 bits.
    |dLSE|: a score is a sum of D products in 32 bits, each addition off by 2^-23 of the
    sum of magnitudes at most: D 2^-23 scale |q||k|, and 2^-21 for the exponentials and the logarithm."""
    scale = cache.D ** -0.5 if scale is None else scale
    ro, rl, spread = ref.attend(q, cache, offsets, scale, causal)
    T = int(offsets[-1])
    rows = slice(int(offsets[0]), T)
    o, lse, ro, rl, spread = o[rows].double(), lse[rows].double(), ro[rows], rl[rows], spread[rows]
    bound = 1.02 * 2.0 ** -8 * (spread + ro.abs()) + 1e-30
    assert torch.isfinite(o).all()
    worst = ((o - ro).abs() / bound).max() if o.numel() else 0.0
    assert worst <= 1, f"O off by {float(worst):.2f} of the bound"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    norm = max((float(k.norm(dim=-1).max()) for k, _ in cache.dense if k.numel()), default=0.0)
    tol = cache.D * 2.0 ** -23 * scale * norm * float(q.float().norm(dim=-1).max()) + 2.0 ** -21 + more
    far = (lse - rl)[~empty].abs() - rl[~empty].abs() * 2.0 ** -23
    assert far.numel() == 0 or float(far.max()) <= tol, (float(far.max()), tol)
    assert attn.attn_get_device_error() == 0


# ----------------------------------------------------------------------------- write, read


def _written(cache, new, seed, stride_heads=0):
    """New tokens k, v of every request (strided slices of one tensor) and what the cache
    holds of them by definition."""
    T = sum(new)
    x = _randn((T, 2 * cache.Hkv + stride_heads, cache.D), seed)
    return x[:, :cache.Hkv], x[:, cache.Hkv:2 * cache.Hkv]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("lens,new", [([1], [1]), ([5, 130, 0, 64, 200], [5, 7, 0, 64, 131]),
                                      ([300, 17], [1, 1]), ([33] * 40, [3] * 40)])
def test_write_and_read(quant, D, page, lens, new):
    Hkv = 3
    c = ref.Cache(lens, Hkv, D, page, quant, seed=1)
    before = [c.kp.clone(), c.vp.clone()]
    scales_before = [c.ks.clone(), c.vs.clone()] if quant else None
    k, v = _written(c, new, 2, stride_heads=1)
    offsets = ref.offsets_of(new)
    attn.cache_write(k, v, c.kp, c.vp, c.table, c.lens_t, offsets, **c.scales())
    out = attn.cache_read(c.kp, c.vp, c.table, c.lens_t, offsets, k.shape[0], **c.scales())
    table = c.table.tolist()
    for x, got, pages, old, i in ((k, out[0], c.kp, before[0], 0), (v, out[1], c.vp, before[1], 1)):
        scale = (c.ks, c.vs)[i] if quant else None
        want_pages = old.clone().view(torch.uint8 if quant else torch.int16)
        want_scale = scales_before[i].clone() if quant else None
        codes, e = ref.quantise(x)
        want = (codes * torch.exp2(e.double()).unsqueeze(-1)).to(BF16) if quant else x
        raw = codes.float().to(E4M3).view(torch.uint8) if quant else x.contiguous().view(torch.int16)
        for b, n in enumerate(new):
            for j in range(n):
                pos, row = lens[b] - n + j, int(offsets[b]) + j
                want_pages[table[b][pos // page], :, pos % page] = raw[row]
                if quant:
                    want_scale[table[b][pos // page], :, pos % page] = (e[row] + 127).to(torch.uint8)
        # the tokens' slots as defined, every other slot as it was
        assert torch.equal(pages.view(want_pages.dtype), want_pages)
        if quant:
            assert torch.equal(scale, want_scale)
        assert torch.equal(got.view(torch.int16), want.contiguous().view(torch.int16))
    assert attn.attn_get_device_error() == 0


def test_write_quantises_every_magnitude():
    """Rows whose largest value runs through the exponents, next to the borders of a scale,
    with subnormal codes, zeros, infinities and NaN."""
    D, page = 64, 16
    rows = []
    for e in range(-126, 128):
        for top in (1.0, 1.75, 1.7578125, 1.9921875):
            x = torch.linspace(-1, 1, D).double() ** 3
            x[5] = top
            rows.append((x * 2.0 ** e).to(BF16))
    n = len(rows)
    special = torch.zeros(4, D, dtype=BF16)
    special[1, 3], special[1, 4] = float("inf"), 1.0
    special[2, 7], special[2, 8] = float("nan"), 2.0
    special[3, 0] = -448.0
    x = torch.cat([torch.stack(rows), special])[:, None].cuda()
    T = x.shape[0]
    P = -(-T // page)
    kp, vp = (torch.zeros(P, 1, page, D, dtype=BF16, device="cuda").to(E4M3) for _ in range(2))
    ks, vs = (torch.zeros(P, 1, page, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    attn.cache_write(x, -x, kp, vp, table, lens, offsets, kscale=ks, vscale=vs)
    k, v = attn.cache_read(kp, vp, table, lens, offsets, T, kscale=ks, vscale=vs)
    codes, e = ref.quantise(x[:n])
    assert torch.equal(ks.reshape(-1)[:n].long(), e.reshape(-1) + 127)
    assert torch.equal(k[:n].double(), codes * torch.exp2(e.double()).unsqueeze(-1))
    assert torch.equal(v[:n], -k[:n])
    s = ks.reshape(-1)[n:].tolist()
    assert s[:1] == [127] and s[1] == 227 and s[2] == 255 and s[3] == 127
    assert not k[n].any()
    assert float(k[n + 1, 0, 3]) == 448 * 2.0 ** 100
    assert torch.isnan(k[n + 2]).all()
    assert float(k[n + 3, 0, 0]) == -448


def test_read_of_every_code_and_scale():
    """256 codes (but e4m3's NaN) under the scales that writing makes."""
    D, page = 128, 64
    values = ref.E4M3_VALUES.clone()
    values[127] = values[255] = 0
    codes = torch.arange(256, dtype=torch.uint8)
    codes[127] = codes[255] = 0
    kp = codes.view(2, 1, 1, D).repeat(101, 1, page, 1).cuda()  # page 2i + j: half j of the codes
    scale = torch.arange(27, 228, dtype=torch.uint8)
    ks = torch.zeros(202, 1, page, dtype=torch.uint8)
    ks[:] = torch.cat([scale, scale[:1]]).view(202, 1, 1)
    ks = ks.cuda()
    table = torch.arange(202, dtype=torch.int32, device="cuda")[None]
    T = 202 * page
    k, v = attn.cache_read(kp.view(E4M3), kp.view(E4M3), table, torch.tensor([T], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, T], dtype=torch.int32, device="cuda"), T, kscale=ks, vscale=ks)
    want = values.view(2, D)[torch.arange(202) % 2] * torch.exp2(ks[:, 0, 0].cpu().double() - 127)[:, None]
    assert torch.equal(k.view(202, page, D).cpu().double(), want[:, None].expand(202, page, D))
    assert torch.equal(k, v)


@pytest.mark.parametrize("quant", [False, True])
def test_tokens_outside_the_cache(quant):
    """More new tokens than the request has, rows of no request, pages out of range."""
    c = ref.Cache([3, 40], 2, 64, 16, quant, seed=3)
    c.table[1, 1] = -5
    offsets = torch.tensor([2, 7, 47], dtype=torch.int32, device="cuda")  # 5 new of 3, 40 of 40
    x = _randn((50, 4, 64), 4)
    before = [c.kp.clone().view(torch.uint8), c.vp.clone().view(torch.uint8)]
    attn.cache_write(x[:, :2], x[:, 2:], c.kp, c.vp, c.table, c.lens_t, offsets, **c.scales())
    assert attn.attn_get_device_error() == 0x40
    k, v = attn.cache_read(c.kp, c.vp, c.table, c.lens_t, offsets, 50, **c.scales())
    assert attn.attn_get_device_error() == 0x40
    for y, z in ((x[:, :2], k), (x[:, 2:], v)):
        if quant:
            codes, e = ref.quantise(y)
            y = (codes * torch.exp2(e.double()).unsqueeze(-1)).to(BF16)
        assert not z[2:4].any()                      # positions -2, -1
        assert torch.equal(z[4:23], y[4:23])         # request 0's three, 1's first page
        assert not z[23:39].any()                    # the page out of range: zeros
        assert torch.equal(z[39:47], y[39:47])
    used = set(c.table[0, :1].tolist() + c.table[1, [0, 2]].tolist())
    for p in range(c.kp.shape[0]):
        if p not in used:
            assert torch.equal(c.kp.view(torch.uint8)[p], before[0][p])
            assert torch.equal(c.vp.view(torch.uint8)[p], before[1][p])


# ----------------------------------------------------------------------------- attention

LENS = [([1], [1]), ([63, 64, 65, 0, 1], [1] * 5), ([1000, 17, 129], [1] * 3),
        ([5, 200, 64, 33, 400], [5, 3, 64, 1, 2]), ([130, 7, 0], [2, 0, 0]), ([600], [600]),
        ([20, 300, 257], [1, 120, 257]), ([2, 40], [6, 40])]


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("lens,new", LENS, ids=[f"{a}-{b}" for a, b in LENS])
@pytest.mark.parametrize("G", [1, 4, 7])
def test_attention(quant, D, page, lens, new, G):
    Hkv = 2
    c = ref.Cache(lens, Hkv, D, page, quant, seed=sum(lens) + page)
    offsets = ref.offsets_of(new)
    q = _randn((sum(new), Hkv * G + 3, D), 7)[:, 1:Hkv * G + 1]
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=max(new), **c.scales())
    check_attention(o, lse, q, c, offsets)
    if all(n == 1 for n in new):
        o, lse = attn.paged_decode(q, *c.args(), **c.scales())
        check_attention(o, lse, q, c, offsets)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 2, 3, 8, 12, 16, 33, 128])
def test_heads(quant, G):
    lens, new = [70, 333], [3, 2]
    c = ref.Cache(lens, 1, 128, 32, quant, seed=G)
    offsets = ref.offsets_of(new)
    q = _randn((5, G, 128), 8)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=3, **c.scales())
    check_attention(o, lse, q, c, offsets)
    o, lse = attn.paged_forward(q, *c.args(), offsets, **c.scales())  # T as the bound
    check_attention(o, lse, q, c, offsets)
    o, lse = attn.paged_decode(q[:2], *c.args(), **c.scales())
    check_attention(o, lse, q[:2], c, ref.offsets_of([1, 1]))


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 4], [40, 200]])
def test_without_the_causal_mask(quant, new):
    c = ref.Cache([50, 210], 2, 64, 16, quant, seed=5)
    offsets = ref.offsets_of(new)
    q = _randn((sum(new), 6, 64), 9)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=max(new), causal=False, scale=0.3, **c.scales())
    check_attention(o, lse, q, c, offsets, causal=False, scale=0.3)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("sigma,scale", [(1.0, 0.0), (8.0, 0.5), (30.0, 1.0), (1e-3, 1.0)])
@pytest.mark.parametrize("new", [1, 90])
def test_steep_and_flat_scores(quant, sigma, scale, new):
    """Scores whose maximum moves with every tile, and those that are all alike."""
    c = ref.Cache([700, 90], 1, 128, 64, quant, seed=6, sigma=sigma)
    offsets = ref.offsets_of([new, new])
    q = _randn((2 * new, 4, 128), 10)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, scale=scale, **c.scales())
    check_attention(o, lse, q, c, offsets, scale=scale)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 70])
def test_rows_of_no_request_are_left_alone(quant, new):
    c = ref.Cache([100, 80], 2, 64, 32, quant, seed=8)
    offsets = ref.offsets_of([new, new], first=3)
    T = 2 * new + 9
    q = _randn((T, 4, 64), 11)
    o = torch.full((T, 4, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((T, 4), 7.0, device="cuda")
    ks, vs = (c.ks, c.vs) if quant else (None, None)
    attn.attn_paged_fwd(q, 4 * 64, c.kp, c.vp, ks, vs, c.table, c.lens_t, offsets, o, lse, 2, T, new, 4, 2,
                        64, 32, c.kp.shape[0], c.table.shape[1], True, 0.125)
    check_attention(o, lse, q, c, offsets)
    for x in (o, lse):
        assert (x[:3] == 7).all() and (x[3 + 2 * new:] == 7).all()


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 50])
def test_pages_out_of_range_read_as_zeros(quant, new):
    c = ref.Cache([100], 1, 64, 16, quant, seed=9)
    for i, bad in ((1, -1), (3, c.kp.shape[0]), (6, 2**31 - 1)):
        c.table[0, i] = bad
        for x in c.dense[0]:
            x[16 * i:16 * i + 16] = 0
    offsets = ref.offsets_of([new])
    q = _randn((new, 2, 64), 12)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    assert attn.attn_get_device_error() == 0x40
    check_attention(o, lse, q, c, offsets)


@pytest.mark.parametrize("new", [1, 70])
def test_scales_of_every_size(new):
    """Rows of K and V whose scales run far apart, the largest of them beyond what one
    factor of bf16 holds."""
    c = ref.Cache([150], 1, 128, 64, True, seed=10)
    k, v = c.dense[0]
    for i in range(150):
        e = (-60, 0, 3, 12, 30, -90)[i % 6]
        at, slot = int(c.table[0, i // 64]), i % 64
        for scale, x, shift in ((c.vs, v, e), (c.ks, k, (0, 9, -20)[i % 3])):
            scale[at, 0, slot] += shift
            x[i] *= 2.0 ** shift
    offsets = ref.offsets_of([new])
    q = _randn((new, 4, 128), 13, sigma=1e-3)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, scale=0.05, **c.scales())
    check_attention(o, lse, q, c, offsets, scale=0.05)


@pytest.mark.parametrize("sigma", [1.0, 1e-8, 1e-25])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("G,new", [(4, 1), (4, 3), (2, 70)])
def test_zeros_beside_small_values(sigma, D, page, G, new):
    """Rows of zeros have the scale 2^0, however small the others are; a query of zeros."""
    lens = [150, 300]
    c = ref.Cache(lens, 1, D, page, True, seed=16, sigma=sigma)
    for b, n in enumerate(lens):
        k, v = c.dense[b]
        for i in [0, 5, 64, 65, n - 1] + list(range(100, 140)):
            at, slot = int(c.table[b, i // page]), i % page
            for pages, scale, x in ((c.kp, c.ks, k), (c.vp, c.vs, v)):
                pages.view(torch.uint8)[at, 0, slot] = 0x80 * (i % 2)
                scale[at, 0, slot] = 127
                x[i] = 0
    offsets = ref.offsets_of([new, new])
    q = _randn((2 * new, G, D), 17)
    q[0] = q[-1, 1:] = 0
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    # The sum of weights is over 2^m with m near the exponents of V's scales, 64 to 128 in
    # magnitude at most: a score less m is rounded by 2^-18, the sum's logarithm is off by 2^-17.
    check_attention(o, lse, q, c, offsets, more=math.log(2) * (2.0 ** -18 + 2.0 ** -17))


@pytest.mark.parametrize("new", [1, 5, 70])
def test_a_nan_reaches_only_its_request(new):
    for quant in (False, True):
        c = ref.Cache([90, 90], 1, 64, 16, quant, seed=11)
        at = int(c.table[0, 0])
        if quant:
            c.ks[at, 0, 3] = 255
        else:
            c.kp[at, 0, 3, 5] = float("nan")
        offsets = ref.offsets_of([new, new])
        q = _randn((2 * new, 2, 64), 14)
        o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
        assert torch.isnan(o[:new]).all() and torch.isnan(lse[:new]).all()
        c.dense[0] = [x[:0] for x in c.dense[0]]
        assert torch.isfinite(o[new:]).all()
        check_attention(o[new:], lse[new:], q[new:], _only(c, 1), ref.offsets_of([new]))


def _only(c, b):
    """The cache as request b sees it."""
    import copy
    d = copy.copy(c)
    d.lens, d.dense = [c.lens[b]], [c.dense[b]]
    return d


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(1, 1), (8, 1), (16, 1), (4, 4)])
def test_long_contexts(quant, D, G, new):
    """So many keys that every CTA goes around its ring many times, next to short requests."""
    lens = [90001, 5, 4, 16384, 900]
    c = ref.Cache(lens, 8, D, 128, quant, seed=12)
    offsets = ref.offsets_of([new] * len(lens))
    q = _randn((new * len(lens), 8 * G, D), 15)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    check_attention(o, lse, q, c, offsets)


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,new", [([9000, 700], [300, 650]), ([2500] * 9, [1] * 8 + [200]),
                                      ([700, 3], [900, 5])])
def test_long_chunks(quant, D, lens, new):
    """Items that are cut between CTAs, at any place."""
    c = ref.Cache(lens, 8, D, 64, quant, seed=13)
    offsets = ref.offsets_of(new)
    q = _randn((sum(new), 24, D), 16)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=max(new), **c.scales())
    check_attention(o, lse, q, c, offsets)
