"""Paged attention over keys and values of very different sizes: what a row does not see, or
sees with next to no weight, costs the others nothing.  Against the definition in 64 bits, with
bounds that count the roundings of each cache type."""
import math

import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402
from attention_forward_sm_gb300 import binding as attn  # noqa: E402
from test_gpu_paged import _randn  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = ref.BF16


def resize(c, b, i, k=0, v=0):
    """Key i of request b: K times 2^k, V times 2^v, by their scales or, in bf16, values."""
    at, slot = int(c.table[b, i // c.page]), i % c.page
    for x, pages, scale, e in ((c.dense[b][0], c.kp, c.ks, k), (c.dense[b][1], c.vp, c.vs, v)):
        x[i] *= 2.0 ** e
        if not c.quant:
            pages[at, :, slot] = x[i].to(BF16)
        elif e:
            scale[at, :, slot] += e


def _exponents(c, b):
    """2^e of the rows of V [n, Hkv] of request b."""
    n = c.lens[b]
    i = torch.arange(n, device="cuda")
    e = c.vs[c.table[b].long()[i // c.page], :, i % c.page].double() - 127
    return torch.where(c.dense[b][1].abs().amax(-1) > 0, e, torch.full_like(e, -100.0))


def check_range(o, lse, q, c, offsets, causal=True, scale=None, only=None):
    """Of every request and head, or of `only` these.  A score is a sum of D products in 32 bits,
    each addition off by 2^-23 of the sum of magnitudes at most: d_j = scale sum_i D 2^-23
    |q_i k_ji|; a query's elements below 2^-14 of its largest are rounded by 2^-25 of that.
    A weight is rounded to bf16 or f16 (half a step 2^-8, 2^-11) and O to bf16 (2^-8); so with
    softmax weights w and everything else in 32 bits (a fiftieth more)
      |dO| <= 2^-8 |O| + sum_j w_j (2^-8 or 2^-11) |v_j| + sum_j w_j d_j (|v_j| + |O|) + floor,
    and n 2^-27 sum_j w_j |v_j| for sums of n products that are cut 26 bits below the highest.
    floor, quantised: half a step of f16 is 2^-25 at least, and the largest product of a weight
    and a scale of V, M = max_j w_j 2^e_j, stands for 2^10 in it, or, since a tile may
    have one scale, for 2^10 over as much as V's scales differ, 2^2 at the least:
    sum_j 2^-35 M min(2^8, max_j 2^e_j / min_j 2^e_j) |code_j|.
    LSE: sum_j w_j d_j, four roundings (score, less the reference, the reference, the end) of
    numbers below |x| + |e| + 64 by 2^-24, 2^-21 for the exponentials and the logarithm."""
    scale = c.D ** -0.5 if scale is None else scale
    off = offsets.tolist()
    G = q.shape[1] // c.Hkv
    half = 2.0 ** -11 if c.quant else 2.0 ** -8
    for b, (k, v) in enumerate(c.dense):
        n, m = off[b + 1] - off[b], c.lens[b]
        rows = slice(off[b], off[b + 1])
        if n == 0 or m == 0:
            continue
        pos = torch.arange(n, device="cuda") + (m - n)
        seen = torch.arange(m, device="cuda")[None] <= (pos[:, None] if causal else m)
        for h in range(q.shape[1]):
            if only and (b, h) not in only:
                continue
            kh, vh, qh = k[:, h // G], v[:, h // G], q[rows, h].double()
            x = (scale * (qh @ kh.T)).masked_fill(~seen, -math.inf)
            rl = torch.logsumexp(x, 1)
            w = torch.exp(x - rl[:, None])
            ro = w @ vh
            most = qh.abs().amax(1, keepdim=True)
            small = (qh != 0) & (qh.abs() < 2.0 ** -14 * most)
            d = w * scale * ((c.D * 2.0 ** -23 * qh.abs() + 2.0 ** -25 * most * small) @ kh.abs().T)
            bound = 2.0 ** -8 * ro.abs() + (half + m * 2.0 ** -27) * (w @ vh.abs()) + d @ vh.abs() + d.sum(1, keepdim=True) * ro.abs()
            far = torch.zeros(n, device="cuda", dtype=torch.float64)
            if c.quant:
                e = _exponents(c, b)[:, h // G]
                top = (w * torch.exp2(e)).amax(1, keepdim=True) * 2.0 ** min(8.0, float(e.max() - e.min()))
                bound += 2.0 ** -35 * top * (seen.double() @ (vh.abs() / torch.exp2(e)[:, None]))
                far += e.abs().amax()
            off_by = (o[rows, h].double() - ro).abs() / (1.02 * bound + 1e-30)
            assert float(off_by.max()) <= 1, (b, h, int(off_by.amax(1).argmax()), float(off_by.max()))
            tol = 1.02 * d.sum(1) + 2.0 ** -21 + 2.0 ** -22 * (x.amax(1).abs() * math.log2(math.e) + far + 64)
            off_by = (lse[rows, h].double() - rl).abs() / tol
            assert float(off_by.max()) <= 1, (b, h, int(off_by.argmax()), float(off_by.max()))
    assert attn.attn_get_device_error() == 0


QUANT = pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
# the kernel for few rows and the one for many
KERNELS = pytest.mark.parametrize("G,new", [(4, 3), (2, 70)])


@QUANT
@KERNELS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_plain_values(quant, G, new, D, page):
    lens = [300, 129, 2000]
    c = ref.Cache(lens, 2, D, page, quant, seed=1)
    offsets = ref.offsets_of([new] * 3)
    q = _randn((3 * new, 2 * G, D), 2)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    check_range(o, lse, q, c, offsets)


@QUANT
@KERNELS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("k,v", [(30, 0), (0, 30), (16, 16), (0, 11)])
def test_unseen_keys_have_no_influence(quant, G, new, D, k, v):
    """The last token's K and V far larger than the others: the rows in front of it do not see
    it (and the row that does is next to orthogonal to it)."""
    lens = [300, 77]
    c = ref.Cache(lens, 1, D, 16, quant, seed=3)
    offsets = ref.offsets_of([new, new])
    q = _randn((2 * new, G, D), 4)
    q[new - 1] = q[2 * new - 1] = 0
    for b, n in enumerate(lens):
        resize(c, b, n - 1, k, v)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    check_range(o, lse, q, c, offsets)


@QUANT
@KERNELS
@pytest.mark.parametrize("e", [12, 15, 22, 30])
@pytest.mark.parametrize("D", [64, 128])
def test_a_large_key_across_the_query(quant, G, new, e, D):
    """A key that is seen by all, large in a dimension that no query has: its score is 0."""
    lens = [300, 90]
    c = ref.Cache(lens, 1, D, 32, quant, seed=5)
    offsets = ref.offsets_of([new, new])
    q = _randn((2 * new, G, D), 6)
    q[..., 0] = 0
    for b in range(2):
        at = int(c.table[b, 0])
        x = torch.zeros(D, device="cuda")
        x[0] = 256.0
        if quant:
            c.kp.view(torch.uint8)[at, 0, 5] = x.to(ref.E4M3).view(torch.uint8)
            c.ks[at, 0, 5] = 127
        c.dense[b][0][5] = x.double()
        resize(c, b, 5, e)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    check_range(o, lse, q, c, offsets)


@QUANT
@KERNELS
@pytest.mark.parametrize("sigma,v", [(1.0, 30), (1.0, 9), (2.0 ** -40, 90)])
def test_large_values_of_little_weight(quant, G, new, sigma, v):
    """A value 2^v times the others', under a weight that leaves nothing of it."""
    lens = [300, 90]
    c = ref.Cache(lens, 1, 64, 64, quant, seed=7)
    offsets = ref.offsets_of([new, new])
    q = _randn((2 * new, G, 64), 8)
    q[..., 0] = 16.0
    for b, n in enumerate(lens):
        for i in range(n):
            resize(c, b, i, 0, round(math.log2(sigma)))
        at = int(c.table[b, 0])
        x = torch.zeros(64, device="cuda")
        x[0] = -64.0  # a score of -128
        if quant:
            c.kp.view(torch.uint8)[at, 0, 9] = x.to(ref.E4M3).view(torch.uint8)
            c.ks[at, 0, 9] = 127
        else:
            c.kp[at, 0, 9] = x.to(BF16)
        c.dense[b][0][9] = x.double()
        resize(c, b, 9, 0, v)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    check_range(o, lse, q, c, offsets)


@QUANT
@KERNELS
@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_decides_a_row(quant, G, new, D):
    """Queries that each select one key, whose sizes run far apart: every row is the value of
    its key, and no other."""
    n = D
    c = ref.Cache([n], 1, D, 16, quant, seed=9)
    k = torch.zeros(n, D, device="cuda")
    k[torch.arange(n), torch.arange(n)] = 8.0
    c.dense[0][0][:] = k.double()[:, None]
    shift = [(0, -60), (9, 0), (-20, 3), (14, 12), (-3, 30), (0, -90), (20, 7)]
    for i in range(n):
        at, slot = int(c.table[0, i // 16]), i % 16
        if quant:
            c.kp.view(torch.uint8)[at, 0, slot] = k[i].to(ref.E4M3).view(torch.uint8)
            c.ks[at, 0, slot] = 127
        resize(c, 0, i, *shift[i % 7])
    for first in range(0, n - new + 1, max(new // 2, 1) * (7 if new < 8 else 1)):
        q = torch.zeros(new, G, D, device="cuda")
        for r in range(new):
            for h in range(G):
                i = (first + r + 3 * h) % n
                q[r, h, i] = 12.5 * 2.0 ** -shift[i % 7][0]  # a score of 100
        q = q.to(BF16)
        offsets = ref.offsets_of([new])
        o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, causal=False, scale=1.0, **c.scales())
        check_range(o, lse, q, c, offsets, causal=False, scale=1.0)


@QUANT
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,G,new", [(20, 4, 1), (1, 20, 240)])
@pytest.mark.parametrize("bits", [20.4, 23.4, 25.4])
def test_many_small_weights_beside_a_large_one(quant, D, B, G, new, bits):
    """A first key that takes nearly all of the weight, but whose value is 0 in all dimensions
    but one, and 2^17 others of 2^-bits of its weight each.  (So many requests or rows that a
    CTA has one from the first key to the last.)"""
    n, Hkv = 2 ** 17 + 77, 8
    c = ref.Cache([n], Hkv, D, 128, quant, seed=11)
    at = int(c.table[0, 0])
    (k, v), dims = c.dense[0], torch.arange(D, device="cuda")
    # the others' scores are 0, their values positive
    k[1:, :, 0] = 0
    k[0] = 64.0 * (dims == 0)
    v.abs_()
    v[0] = 3.5 * (dims == 0)
    if quant:
        c.kp.view(torch.uint8)[..., 0] = 0
        c.vp.view(torch.uint8).bitwise_and_(0x7F)
        for x, pages, scale in ((k, c.kp, c.ks), (v, c.vp, c.vs)):
            pages.view(torch.uint8)[at, :, 0] = (x[0] * 64).float().clamp(max=448).to(ref.E4M3).view(torch.uint8)
            scale[at, :, 0] = 127 - 6
        k[0] = 7.0 * (dims == 0)
    else:
        c.kp[..., 0] = 0
        c.vp.abs_()
        c.kp[at, :, 0], c.vp[at, :, 0] = k[0].to(BF16), v[0].to(BF16)
    # requests that share their pages
    c.table, c.lens_t = c.table.repeat(B, 1), c.lens_t.repeat(B)
    c.lens, c.dense = c.lens * B, c.dense * B
    q = torch.zeros(B * new, Hkv * G, D, device="cuda")
    q[..., 0] = bits * math.log(2) / float(k[0, 0, 0])
    q = q.to(BF16)
    offsets = ref.offsets_of([new] * B)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, scale=1.0, **c.scales())
    check_range(o, lse, q, c, offsets, scale=1.0, only=((0, 0), (B - 1, Hkv * G - 1)))


@KERNELS
@pytest.mark.parametrize("spread", [(-100, 60), (60, -100), (-100, -100), (-50, 70)])
def test_lse_knows_nothing_of_values(G, new, spread):
    """Scales of V as far apart as they get, between tiles and within them."""
    lens = [500, 200]
    c = ref.Cache(lens, 1, 64, 64, True, seed=13)
    offsets = ref.offsets_of([new, new])
    q = _randn((2 * new, G, 64), 14)
    for b, n in enumerate(lens):
        for i in range(n):
            at, slot = int(c.table[b, i // 64]), i % 64
            e = spread[i // 128 % 2] if b == 0 else spread[i % 2]
            c.dense[b][1][i] *= 2.0 ** (e + 127 - int(c.vs[at, 0, slot]))
            c.vs[at, 0, slot] = e + 127
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    check_range(o, lse, q, c, offsets)


@KERNELS
@pytest.mark.parametrize("n", [130, 40000])
def test_values_of_zeros(G, new, n):
    """A cache whose V is all zeros: O is 0, LSE as ever."""
    c = ref.Cache([n], 1, 64, 128, True, seed=15)
    c.vp.view(torch.uint8).bitwise_and_(0x80)
    c.vs.fill_(127)
    c.dense[0][1].zero_()
    offsets = ref.offsets_of([new])
    q = _randn((new, G, 64), 16)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
    assert not o.any()
    check_range(o, lse, q, c, offsets)


@KERNELS
@pytest.mark.parametrize("sigma", [1.0, 1e-8, 1e-25])
@pytest.mark.parametrize("zeros", [range(0, 256), range(256, 384), range(500, 700)])
def test_tiles_of_zeros_beside_small_values(G, new, sigma, zeros):
    """Whole tiles of keys whose V is zeros and says 2^0."""
    n = 700
    c = ref.Cache([n], 1, 64, 64, True, seed=17, sigma=sigma)
    up = -round(math.log2(sigma))  # K as large as ever
    c.dense[0][0].mul_(2.0 ** up)
    c.ks += up
    for x in c.dense[0]:
        x[list(zeros)] = 0
    for i in zeros:
        at, slot = int(c.table[0, i // 64]), i % 64
        for pages, scale in ((c.kp, c.ks), (c.vp, c.vs)):
            pages.view(torch.uint8)[at, :, slot] = 0x80 * (i % 2)
            scale[at, :, slot] = 127
    offsets = ref.offsets_of([new])
    q = _randn((new, G, 64), 18)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, causal=False, **c.scales())
    check_range(o, lse, q, c, offsets, causal=False)


@pytest.mark.parametrize("G,new,lens", [(4, 3, [9000, 130]), (2, 70, [300, 4000]), (3, 300, [9000, 700]), (16, 40, [1500, 41])])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("causal", [True, False])
def test_scales_at_random(G, new, lens, D, page, causal):
    """Runs of ordinary tokens and of tokens with scales of any size, items cut anywhere; pages out
    of range and a key of NaN that only the last rows see."""
    c = ref.Cache(lens, 2, D, page, True, seed=sum(lens) + D)
    g = torch.Generator().manual_seed(page + new)
    offsets = ref.offsets_of([new] * len(lens))
    q = _randn((new * len(lens), 2 * G, D), 19)
    for b, n in enumerate(lens):
        i = torch.arange(n)
        wild = (torch.rand(n // 100 + 1, generator=g) < 0.4)[i // 100]
        at, slot = c.table[b].long()[(i // page).cuda()], (i % page).cuda()
        for x, scale, lo, hi in ((c.dense[b][0], c.ks, -24, 1), (c.dense[b][1], c.vs, -30, 31)):
            e = torch.randint(lo, hi, (n,), generator=g) * wild
            x *= torch.exp2(e.double()).cuda()[:, None, None]
            scale[at, :, slot] += e.to(torch.uint8).cuda()[:, None]  # (modulo 256)
    bad = lens[0] // page // 2
    c.table[0, bad] = -1
    for x in c.dense[0]:
        x[bad * page:(bad + 1) * page] = 0
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=new, causal=causal, **c.scales())
    assert attn.attn_get_device_error() == 0x40
    check_range(o, lse, q, c, offsets, causal=causal)
    if causal:  # the last token's K NaN: nothing for those in front
        for b, n in enumerate(lens):
            c.ks[int(c.table[b, (n - 1) // page]), :, (n - 1) % page] = 255
        o2, lse2 = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
        assert attn.attn_get_device_error() == 0x40
        for b in range(len(lens)):
            last = (b + 1) * new - 1
            assert torch.isnan(o2[last]).all() and torch.isnan(lse2[last]).all()
            o2[last], lse2[last] = o[last], lse[last]
        check_range(o2, lse2, q, c, offsets)
