"""Attention with modified scores on the GPU: forward_mod, row_ranges,
decode_varlen and decode_prefix against the definition in 64 bits.

Tolerances, from the roundings (none measured).  A score x is a product of D
terms summed in fp32 (each step off by one unit, 2^-23, of the sum of the
terms' magnitudes S), scaled, capped (the tanh is good to 2^-20 of the value,
a few roundings more) and biased (roundings of the bias relative to the
nearest key); its error is at most
    dx = (D + 4) 2^-23 S + 2^-19 |x| + 2^-22 |bias|,
and a weight exp(x - LSE) is off by 2 dx + 2^-20 of its value.  The weights
are rounded to bf16 (half a step: 2^-8), and so is O:
    |dO| <= (2^-8 + 2 dx + 2^-19) sum_j w_j |v_j| + 2^-8 |O| + 2^-133
(the last: half the smallest bf16),  |dLSE| <= dx + 2^-19 + 2^-22 |LSE|.

The sums over n keys add at most 64 weights to one another and those sums in
turn, n / 64 + 64 additions in a chain; every addition of positive terms is
off by 2^-24 of the sum at most, which adds (n / 64 + 64) 2^-24 to the
relative error of the normaliser (to dLSE) and, with that of the sum of the
values, twice that to the weights of O.
"""
import math

import pytest
import torch

from attention_forward_sm_gb300 import binding as attn

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _library():
    from attention_forward_sm_gb300 import _build
    _build.build()
    attn.load()
    assert torch.cuda.is_available(), "gpu tests need a CUDA device"


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    assert attn.attn_get_device_error() == 0


def rand(seed, shape, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def alibi(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


def definition(q, k, v, pos, jpos, seen, scale, cap, slope):
    """One head in 64 bits: q [R, D], k / v [n, D], seen [R, n] ->
    O, LSE and the tolerances of both."""
    D = q.shape[1]
    scale = float(torch.tensor(scale, dtype=torch.float32))
    q, k, v = q.double(), k.double(), v.double()
    # keys that no row sees may hold anything
    used = seen.any(0)
    k, v = torch.where(used[:, None], k, 0.0), torch.where(used[:, None], v, 0.0)
    x = scale * (q @ k.T)
    mag = scale * (q.abs() @ k.abs().T)
    if cap > 0:
        cap = float(torch.tensor(cap, dtype=torch.float32))
        x = cap * torch.tanh(x / cap)
    bias = torch.zeros_like(x)
    if slope is not None:
        bias = -float(slope) * (pos.double()[:, None] - jpos.double()[None, :]).abs()
    best = bias.masked_fill(~seen, -INF).amax(1, keepdim=True)
    dx = (D + 4) * 2.0**-23 * mag + 2.0**-19 * x.abs() + 2.0**-22 * (bias - best).abs()
    dx = torch.where(seen, dx, 0.0).amax(1)
    x = (x + bias).masked_fill(~seen, -INF)
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    o = w @ v
    sums = (k.shape[0] / 64 + 64) * 2.0**-24
    tol_o = (2.0**-8 + 2 * dx[:, None] + 2 * sums + 2.0**-19) * (w @ v.abs()) + 2.0**-8 * o.abs() + 2.0**-133
    tol_l = dx + sums + 2.0**-19 + 2.0**-22 * lse.abs()
    return o, lse, tol_o, tol_l


def check(o, lse, ref, label=""):
    ro, rl, to, tl = ref
    none = torch.isinf(rl)
    assert torch.equal(lse.double() == -INF, none), f"{label}: rows that see nothing"
    assert (o[none] == 0).all(), f"{label}: O of rows that see nothing"
    eo = ((o.double() - ro).abs() / to)[~none]
    el = ((lse.double() - rl).abs() / tl)[~none]
    assert not eo.numel() or eo.max() <= 1, f"{label}: O off by {eo.max():.3g} tolerances"
    assert not el.numel() or el.max() <= 1, f"{label}: LSE off by {el.max():.3g} tolerances"


def check_fwd(o, lse, q, k, v, causal, scale, cap, slopes, ranges, q_offset, label=""):
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    pos = q_offset + torch.arange(Nq, device="cuda")
    j = torch.arange(Nk, device="cuda")
    for b in range(B):
        seen = torch.ones(Nq, Nk, dtype=torch.bool, device="cuda")
        if ranges is not None:
            seen &= (j >= ranges[b, :, :1]) & (j < ranges[b, :, 1:])
        if causal:
            seen &= j <= pos[:, None]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            ref = definition(q[b, h], k[b, g], v[b, g], pos, j, seen, scale, cap,
                             None if slopes is None else slopes[h])
            check(o[b, h], lse[b, h], ref, f"{label} b{b} h{h}")


def ranges_of(kind, B, Nq, Nk, seed=5):
    if kind is None:
        return None
    if kind == "docs":
        cut = max(1, Nq // 3)
        lens = torch.tensor([[cut, 0, 1, Nq - cut - 1 - Nq // 7]] * B, dtype=torch.int32, device="cuda")
        return attn.row_ranges(lens, Nq)
    if kind == "prefix":
        lens = torch.tensor([[Nq // 2, Nq - Nq // 2]] * B, dtype=torch.int32, device="cuda")
        return attn.row_ranges(lens, Nq, prefix_lens=lens // 3)
    if kind == "none":
        return torch.zeros(B, Nq, 2, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randint(-5, Nk + 6, (B, Nq, 2), generator=g, device="cuda", dtype=torch.int32)
    if kind == "wild":  # out of range on both sides, lo > hi, and the extremes of the type
        a[:, ::7, 0], a[:, ::7, 1] = -2**31, 2**31 - 1
        a[:, 3::11, 0], a[:, 3::11, 1] = 2**31 - 1, -2**31
        return a
    width = 40
    lo = a[..., 0].clamp(0, Nk)
    return torch.stack([lo, (lo + width).clamp(max=Nk)], -1).contiguous()  # "narrow"


# ------------------------------------------------------------------------------ prefill

FWD = [
    # B, Hq, Hkv, Nq, Nk, D, causal, q_offset, cap, bias, ranges
    (1, 1, 1, 1, 1, 64, False, 0, 0.0, False, None),
    (1, 1, 1, 1, 1, 128, True, 0, 30.0, True, None),
    (2, 2, 2, 256, 256, 64, True, 0, 30.0, False, None),
    (1, 4, 2, 300, 300, 128, True, 0, 50.0, False, None),
    (1, 4, 2, 300, 300, 128, False, 0, 50.0, False, None),
    (2, 4, 1, 257, 385, 64, False, 0, 0.0, True, None),
    (1, 3, 1, 130, 517, 128, True, 387, 0.0, True, None),
    (1, 7, 1, 129, 127, 128, True, 0, 20.0, True, None),
    (2, 2, 1, 511, 511, 128, False, 0, 0.0, False, "docs"),
    (2, 2, 2, 640, 640, 64, False, 0, 25.0, False, "docs"),
    (1, 6, 2, 400, 400, 128, False, 0, 30.0, True, "prefix"),
    (1, 2, 2, 333, 333, 64, False, 0, 0.0, True, "prefix"),
    (2, 2, 1, 300, 450, 128, False, 0, 0.0, False, "wild"),
    (2, 2, 1, 300, 450, 64, True, 100, 15.0, True, "wild"),
    (1, 2, 2, 1000, 900, 128, False, 0, 0.0, False, "narrow"),
    (1, 2, 2, 700, 2000, 64, False, 0, 40.0, True, "narrow"),
    (1, 2, 1, 270, 140, 128, False, 0, 0.0, True, "none"),
    (1, 2, 1, 5, 4099, 128, True, 4094, 30.0, True, None),
    (1, 1, 1, 1030, 1030, 64, True, 0, 0.0, False, "wild"),
]


@pytest.mark.parametrize("case", FWD, ids=lambda c: "-".join(map(str, c)))
def test_forward_mod(case):
    B, Hq, Hkv, Nq, Nk, D, causal, off, cap, bias, kind = case
    q, k, v = (rand(s, sh, sg) for s, sh, sg in ((1, (B, Hq, Nq, D), 6.0 if cap else 1.0),
                                                 (2, (B, Hkv, Nk, D), 1.0), (3, (B, Hkv, Nk, D), 1.0)))
    slopes, ranges = (alibi(Hq) if bias else None), ranges_of(kind, B, Nq, Nk)
    args = dict(causal=causal, softcap=cap, slopes=slopes, ranges=ranges, q_offset=off)
    o, lse = attn.forward_mod(q, k, v, **args)
    check_fwd(o, lse, q, k, v, causal, 1 / math.sqrt(D), cap, slopes, ranges, off)
    o2, lse2 = attn.forward_mod(q, k, v, **args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # the same bits every time


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sigma,cap", [(40.0, 5.0), (200.0, 50.0), (0.01, 1000.0), (1.0, 0.05), (6.0, 50.0)])
def test_cap_over_its_whole_range(D, sigma, cap):
    """Scores far beyond the cap, near its knee and far below it."""
    q, k, v = rand(1, (1, 2, 200, D), sigma), rand(2, (1, 2, 300, D)), rand(3, (1, 2, 300, D))
    o, lse = attn.forward_mod(q, k, v, softcap=cap)
    check_fwd(o, lse, q, k, v, False, 1 / math.sqrt(D), cap, None, None, 0)


@pytest.mark.parametrize("slope", [0.5, -0.01, 8.0, 0.0])
@pytest.mark.parametrize("q_offset", [0, 150, 10**6, 2_000_000_000])
def test_bias_of_far_positions(slope, q_offset):
    """The bias keeps its digits when every key is far away: it is taken
    relative to the key that it favours."""
    D, Nq, Nk = 64, 70, 300
    q, k, v = rand(1, (1, 2, Nq, D)), rand(2, (1, 1, Nk, D)), rand(3, (1, 1, Nk, D))
    slopes = torch.tensor([slope, slope / 3], device="cuda")
    o, lse = attn.forward_mod(q, k, v, slopes=slopes, q_offset=q_offset)
    check_fwd(o, lse, q, k, v, False, 1 / math.sqrt(D), 0.0, slopes, None, q_offset)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [1e-30, 1e-7, 1e-3, 0.3, 1e4, 1e12, 1e30])
@pytest.mark.parametrize("bias", [False, True])
def test_caps_far_from_the_scores_in_masked_tiles(D, cap, bias):
    """Caps for which some polynomials, or all, cannot be formed in fp32; scores of
    0 too; rows that see a part of a tile, with anything at the keys they do not see."""
    q, k, v = rand(1, (1, 2, 200, D)), rand(2, (1, 1, 300, D)), rand(3, (1, 1, 300, D))
    k[:, :, 40:60] = 0
    k[:, :, 291:] = 1e30
    ranges = torch.tensor([[[i % 97, min(290, i + 50)] for i in range(200)]], dtype=torch.int32, device="cuda")
    slopes = torch.tensor([0.1, 0.01], device="cuda") if bias else None
    o, lse = attn.forward_mod(q, k, v, softcap=cap, slopes=slopes, ranges=ranges)
    check_fwd(o, lse, q, k, v, False, 1 / math.sqrt(D), cap, slopes, ranges, 0)
    lens = torch.tensor([290], dtype=torch.int32, device="cuda")
    o, lse = attn.decode_varlen(q[:, :, 0].contiguous(), k, v, lens, softcap=cap, slopes=slopes)
    check_decode(o, lse, q[:, :, 0], k, v, [290], cap, slopes)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0, 0.5])
@pytest.mark.parametrize("kind", [None, "wild", "prefix"])
def test_bias_of_keys_on_both_sides(D, cap, kind):
    """Slopes of either sign, shallow and steep, for rows that see keys on both sides
    of their position, on one side, or none; scores within the cap and far beyond."""
    q, k, v = rand(1, (1, 6, 260, D), 2.0), rand(2, (1, 2, 390, D)), rand(3, (1, 2, 390, D))
    slopes = torch.tensor([0.02, -0.02, 0.9, -0.9, 6.0, 0.0], device="cuda")
    r = ranges_of(kind, 1, 260, 390) if kind else None
    o, lse = attn.forward_mod(q, k, v, softcap=cap, slopes=slopes, ranges=r, q_offset=60)
    check_fwd(o, lse, q, k, v, False, 1 / math.sqrt(D), cap, slopes, r, 60)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, False), (30.0, True)])
@pytest.mark.parametrize("trash", [NAN, INF, -INF])
def test_trash_in_keys_that_no_row_sees(D, cap, bias, trash):
    """K and V of padding (in front of and behind the visible span, inside and
    outside of the key tiles that are read) have no influence."""
    B, N, lo, hi = 2, 400, 37, 301
    q, k, v = rand(1, (B, 2, N, D)), rand(2, (B, 1, N, D)), rand(3, (B, 1, N, D))
    ranges = torch.tensor([lo, hi], dtype=torch.int32, device="cuda").expand(B, N, 2).contiguous()
    for x in (k, v):
        x[:, :, :lo] = trash
        x[:, :, hi:] = trash
    slopes = alibi(2) if bias else None
    o, lse = attn.forward_mod(q, k, v, softcap=cap, slopes=slopes, ranges=ranges)
    check_fwd(o, lse, q, k, v, False, 1 / math.sqrt(D), cap, slopes, ranges, 0)


def test_nan_in_k_reaches_only_the_rows_that_see_it():
    N, D = 300, 128
    q, k, v = rand(1, (1, 1, N, D)), rand(2, (1, 1, N, D)), rand(3, (1, 1, N, D))
    k[0, 0, 200] = NAN
    o, lse = attn.forward_mod(q, k, v, causal=True, softcap=30.0)
    assert torch.isfinite(o[0, 0, :200].float()).all() and torch.isfinite(lse[0, 0, :200]).all()
    assert torch.isnan(o[0, 0, 200:].float()).all() and torch.isnan(lse[0, 0, 200:]).all()


def test_without_modifications_it_is_forward():
    for D in (64, 128):
        q, k, v = rand(1, (2, 4, 600, D)), rand(2, (2, 2, 700, D)), rand(3, (2, 2, 700, D))
        for causal in (False, True):
            o, lse = attn.forward_mod(q, k, v, causal=causal)
            ro, rl = attn.forward(q, k, v, causal=causal)
            # both within the tolerance of the definition: within twice that of one another
            assert (o.float() - ro.float()).abs().max() <= 2 * 2.0**-6
            assert (lse - rl).abs().max() <= 1e-4


def test_scale_zero_and_large():
    q, k, v = rand(1, (1, 2, 150, 64)), rand(2, (1, 2, 150, 64)), rand(3, (1, 2, 150, 64))
    for scale in (0.0, 3.0):
        for cap in (0.0, 20.0):
            o, lse = attn.forward_mod(q, k, v, scale=scale, softcap=cap, causal=True)
            check_fwd(o, lse, q, k, v, True, scale, cap, None, None, 0)


def test_many_units_every_row():
    """More work units than CTAs, of very different lengths, every row checked."""
    B, H, N, D = 3, 24, 1100, 128
    q, k, v = rand(1, (B, H, N, D)), rand(2, (B, H, N, D)), rand(3, (B, H, N, D))
    lens = torch.tensor([[1, 300, 2, 500, 97, 130], [1100, 0, 0, 0, 0, 0], [7, 7, 400, 600, 0, 0]],
                        dtype=torch.int32, device="cuda")
    ranges = attn.row_ranges(lens, N)
    o, lse = attn.forward_mod(q, k, v, ranges=ranges, softcap=12.0)
    check_fwd(o, lse, q, k, v, False, 1 / math.sqrt(D), 12.0, None, ranges, 0)


# ------------------------------------------------------------------------------ ranges


def ranges_definition(doc_lens, prefix, N, causal):
    out = torch.zeros(len(doc_lens), N, 2, dtype=torch.int32)
    for b, row in enumerate(doc_lens):
        s = 0
        for m, n in enumerate(row):
            e = min(s + max(n, 0), N)
            for i in range(s, e):
                hi = e if not causal else max(i + 1, min(s + (max(prefix[b][m], 0) if prefix else 0), e))
                out[b, i] = torch.tensor([s, hi])
            s = e
    return out


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("rows,N", [
    ([[1]], 1), ([[5]], 3), ([[0]], 4), ([[-3, 2, 0, 0, 4]], 9), ([[2, 3], [6, 0], [0, 6]], 6),
    ([[1023, 2, 1024]], 2100), ([[1] * 1500], 1400), ([[0] * 1100 + [3] * 1100], 3000),
    ([[2**31 - 1, 5], [3, 2**31 - 1]], 1030),
])
def test_row_ranges(rows, N, causal):
    lens = torch.tensor(rows, dtype=torch.int32, device="cuda")
    pre = [[(7 * m) % 5 - 1 if m % 3 else 2**31 - 1 for m in range(len(r))] for r in rows]
    for prefix in (None, pre):
        t = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda")
        got = attn.row_ranges(lens, N, prefix_lens=t, causal=causal)
        assert torch.equal(got.cpu(), ranges_definition(rows, prefix, N, causal))


# ------------------------------------------------------------------------------ decode


def check_decode(o, lse, q, k, v, lens, cap, slopes, pk=None, pv=None, scale=None, rows=None):
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    for b in range(B) if rows is None else rows:
        n = lens[b]
        for g in range(Hkv):
            kk, vv = k[b, g, :n], v[b, g, :n]
            if pk is not None:
                kk, vv = torch.cat([pk[g], kk]), torch.cat([pv[g], vv])
            heads = range(g * G, (g + 1) * G)
            if kk.shape[0] == 0:
                assert (o[b, list(heads)] == 0).all() and (lse[b, list(heads)] == -INF).all()
                continue
            j = torch.arange(kk.shape[0], device="cuda")
            seen = torch.ones(1, kk.shape[0], dtype=torch.bool, device="cuda")
            for h in heads:
                ref = definition(q[b, h:h + 1], kk, vv, j[-1:], j, seen,
                                 1 / math.sqrt(D) if scale is None else scale, cap,
                                 None if slopes is None else slopes[h])
                check(o[b, h:h + 1], lse[b, h:h + 1], ref, f"b{b} h{h} len {n}")


DECODE = [
    # Hq, Hkv, Ncap, D, cap, bias, lens
    (1, 1, 1, 64, 0.0, False, [1]),
    (2, 1, 1, 128, 30.0, True, [1, 0]),
    (4, 2, 300, 128, 0.0, False, [0, 1, 2, 127, 128, 129, 255, 256, 257, 300]),
    (8, 2, 513, 64, 40.0, True, [513, 0, 64, 65, 384]),
    (32, 8, 1023, 128, 50.0, False, [1023]),
    (14, 2, 700, 64, 0.0, True, [700, 3, 511]),
    (6, 2, 260, 128, 25.0, True, [260, 1]),
    (16, 1, 400, 128, 0.0, False, [333, 400]),
    (64, 1, 200, 64, 30.0, False, [199, 0, 130]),
    (128, 1, 129, 128, 30.0, True, [129, 128]),
    (40, 2, 140, 128, 0.0, True, [140, 17]),
    (4, 4, 20000, 128, 50.0, False, [20000, 5, 9000]),
    (8, 1, 40000, 64, 0.0, True, [40000, 39]),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c[:6])) + f"-B{len(c[6])}")
def test_decode_varlen(case):
    Hq, Hkv, Ncap, D, cap, bias, lens = case
    B = len(lens)
    q, k, v = rand(1, (B, Hq, D), 6.0 if cap else 1.0), rand(2, (B, Hkv, Ncap, D)), rand(3, (B, Hkv, Ncap, D))
    for b, n in enumerate(lens):  # the unused tail may hold anything
        for x in (k, v):
            x[b, :, n:] = (NAN, INF, -INF)[b % 3]
    slopes = alibi(Hq) if bias else None
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_varlen(q, k, v, t, softcap=cap, slopes=slopes)
    check_decode(o, lse, q, k, v, lens, cap, slopes)
    o2, lse2 = attn.decode_varlen(q, k, v, t, softcap=cap, slopes=slopes)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_varlen_clamps_lengths_and_takes_none():
    q, k, v = rand(1, (3, 4, 64)), rand(2, (3, 2, 200, 64)), rand(3, (3, 2, 200, 64))
    t = torch.tensor([-7, 2**31 - 1, -2**31], dtype=torch.int32, device="cuda")
    o, lse = attn.decode_varlen(q, k, v, t)
    check_decode(o, lse, q, k, v, [0, 200, 0], 0.0, None)
    o, lse = attn.decode_varlen(q, k, v)
    check_decode(o, lse, q, k, v, [200] * 3, 0.0, None)


def test_decode_varlen_is_decode():
    q, k, v = rand(1, (2, 8, 128)), rand(2, (2, 2, 999, 128)), rand(3, (2, 2, 999, 128))
    o, lse = attn.decode_varlen(q, k, v)
    ro, rl = attn.decode(q, k, v, nsplit=4)
    assert (o.float() - ro.float()).abs().max() <= 2.0**-6 and (lse - rl).abs().max() <= 1e-4


PREFIX = [
    # Hq, Hkv, Np, Ncap, D, cap, bias, lens
    (1, 1, 1, 1, 64, 0.0, False, [0]),
    (2, 1, 1, 4, 128, 30.0, True, [4, 0, 1]),
    (4, 2, 128, 130, 128, 0.0, False, [0, 1, 128, 129, 130]),
    (8, 1, 1001, 200, 64, 0.0, True, [1, 200, 50, 0, 77]),
    (32, 8, 700, 150, 128, 50.0, False, list(range(0, 150, 4))),
    (7, 1, 513, 40, 64, 30.0, True, [40, 0, 13] * 13),       # 7 heads: 18 requests to a query tile
    (12, 4, 400, 64, 128, 0.0, False, [64, 1] * 50),         # 3 heads, 42 requests to a tile
    (80, 1, 300, 20, 128, 20.0, False, [20, 3, 0, 9]),       # a tile holds one request
    (128, 1, 200, 129, 64, 0.0, True, [129, 0, 5]),
    (16, 2, 5000, 300, 128, 0.0, False, [300, 20] * 40),
    (4, 1, 20000, 10, 64, 40.0, True, [10, 0]),
]


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c[:7])) + f"-B{len(c[7])}")
def test_decode_prefix(case):
    Hq, Hkv, Np, Ncap, D, cap, bias, lens = case
    B = len(lens)
    q = rand(1, (B, Hq, D), 6.0 if cap else 1.0)
    k, v = rand(2, (B, Hkv, Ncap, D)), rand(3, (B, Hkv, Ncap, D))
    pk, pv = rand(4, (Hkv, Np, D)), rand(5, (Hkv, Np, D))
    for b, n in enumerate(lens):
        for x in (k, v):
            x[b, :, n:] = (NAN, INF, -INF)[b % 3]
    slopes = alibi(Hq) if bias else None
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_prefix(q, pk, pv, k, v, t, softcap=cap, slopes=slopes)
    check_decode(o, lse, q, k, v, lens, cap, slopes, pk, pv)
    o2, lse2 = attn.decode_prefix(q, pk, pv, k, v, t, softcap=cap, slopes=slopes)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("slope", [0.25, -0.25])
def test_decode_bias_of_both_signs(slope):
    lens = [900, 0, 3]
    q, k, v = rand(1, (3, 4, 64)), rand(2, (3, 2, 900, 64)), rand(3, (3, 2, 900, 64))
    pk, pv = rand(4, (2, 3000, 64)), rand(5, (2, 3000, 64))
    slopes = torch.tensor([slope, -slope, slope / 50, 0.0], device="cuda")
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_prefix(q, pk, pv, k, v, t, slopes=slopes)
    check_decode(o, lse, q, k, v, lens, 0.0, slopes, pk, pv)
    o, lse = attn.decode_varlen(q, k, v, t, slopes=slopes)
    check_decode(o, lse, q, k, v, lens, 0.0, slopes)


def test_many_requests():
    B, Hq, Hkv, D, Ncap = 700, 4, 2, 64, 33
    lens = [(17 * b) % 34 for b in range(B)]
    q, k, v = rand(1, (B, Hq, D)), rand(2, (B, Hkv, Ncap, D)), rand(3, (B, Hkv, Ncap, D))
    pk, pv = rand(4, (Hkv, 129, D)), rand(5, (Hkv, 129, D))
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_varlen(q, k, v, t)
    check_decode(o, lse, q, k, v, lens, 0.0, None, rows=range(0, B, 9))
    o, lse = attn.decode_prefix(q, pk, pv, k, v, t)
    check_decode(o, lse, q, k, v, lens, 0.0, None, pk, pv, rows=range(0, B, 9))


def test_cache_offsets_beyond_32_bits():
    B, Hkv, Ncap, D = 3, 2, 3_000_000, 128  # 2.3e9 elements, 4.6e9 bytes per cache
    k = torch.zeros(B, Hkv, Ncap, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    lens = [5, 100, 300]
    for b, n in enumerate(lens):
        k[b, :, :n] = rand(10 + b, (Hkv, n, D))
        v[b, :, :n] = rand(20 + b, (Hkv, n, D))
    q = rand(1, (B, 4, D))
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_varlen(q, k, v, t)
    check_decode(o, lse, q, k, v, lens, 0.0, None)
    # a cache that is full to its end
    t = torch.tensor([0, 0, Ncap], dtype=torch.int32, device="cuda")
    k[2, 1, Ncap - 300:] = rand(30, (300, D))
    v[2, 1, Ncap - 300:] = rand(31, (300, D))
    o, lse = attn.decode_varlen(q, k, v, t)
    check_decode(o, lse, q, k, v, [0, 0, Ncap], 0.0, None, rows=[2])


# ------------------------------------------------------------------------------ together


def test_a_prompt_then_tokens_as_a_server_runs_them():
    """Packed prompts through row_ranges and forward_mod, then decode steps on
    caches that grow, with and without sharing the prompt: every step is the
    last row of a prefill of the same tokens."""
    Hq, Hkv, D, cap, P, T = 8, 2, 128, 30.0, 210, 4
    slopes = alibi(Hq)
    q, k, v = rand(1, (1, Hq, P + T, D), 4.0), rand(2, (1, Hkv, P + T, D)), rand(3, (1, Hkv, P + T, D))
    lens = torch.tensor([[P + T]], dtype=torch.int32, device="cuda")
    whole, wl = attn.forward_mod(q, k, v, softcap=cap, slopes=slopes,
                                 ranges=attn.row_ranges(lens, P + T))
    # the prompt in two chunks
    for a, b in ((0, 100), (100, P)):
        o, l = attn.forward_mod(q[:, :, a:b].contiguous(), k[:, :, :b].contiguous(),
                                v[:, :, :b].contiguous(), causal=True, q_offset=a, softcap=cap,
                                slopes=slopes)
        assert (o.float() - whole[:, :, a:b].float()).abs().max() <= 2.0**-5
        assert (l - wl[:, :, a:b]).abs().max() <= 1e-4
    kc = torch.full((1, Hkv, 300, D), NAN, dtype=torch.bfloat16, device="cuda")
    vc, ks, vs = kc.clone(), kc.clone(), kc.clone()
    kc[:, :, :P], vc[:, :, :P] = k[:, :, :P], v[:, :, :P]
    for t in range(T):
        kc[:, :, P + t], vc[:, :, P + t] = k[:, :, P + t], v[:, :, P + t]
        ks[:, :, t], vs[:, :, t] = k[:, :, P + t], v[:, :, P + t]
        q1 = q[:, :, P + t].contiguous()
        n = torch.tensor([P + t + 1], dtype=torch.int32, device="cuda")
        for o, l in (attn.decode_varlen(q1, kc, vc, n, softcap=cap, slopes=slopes),
                     attn.decode_prefix(q1, k[0, :, :P].contiguous(), v[0, :, :P].contiguous(), ks, vs,
                                        n - P, softcap=cap, slopes=slopes)):
            assert (o.float() - whole[:, :, P + t].float()).abs().max() <= 2.0**-5
            assert (l - wl[:, :, P + t]).abs().max() <= 1e-4


def _busy(s):
    with torch.cuda.stream(s):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-4
    return a


def test_calls_on_other_streams_at_once():
    """Two streams that run the calls at the same time, one of them named by
    its handle; scratch is never shared between them."""
    sets = []
    for i in range(2):
        lens = [500 - 90 * i, 3, 77 + i]
        sets.append((rand(i, (3, 8, 64)), rand(10 + i, (3, 2, 500, 64)), rand(20 + i, (3, 2, 500, 64)),
                     rand(30 + i, (2, 900, 64)), rand(40 + i, (2, 900, 64)), lens,
                     torch.tensor(lens, dtype=torch.int32, device="cuda")))
    x = rand(50, (1, 2, 300, 64))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for r in range(6):
        for i, s in enumerate(streams):
            q, k, v, pk, pv, lens, t = sets[i]
            h = s if i else s.cuda_stream
            outs.append((i, True, attn.decode_prefix(q, pk, pv, k, v, t, stream=h)))
            outs.append((i, False, attn.decode_varlen(q, k, v, t, stream=h)))
    f = attn.forward_mod(x, x, x, causal=True, stream=streams[0])
    torch.cuda.synchronize()
    for i, prefix, (o, lse) in outs:
        q, k, v, pk, pv, lens, t = sets[i]
        check_decode(o, lse, q, k, v, lens, 0.0, None, *((pk, pv) if prefix else ()))
    check_fwd(*f, x, x, x, True, 1 / 8, 0.0, None, None, 0)


def test_inputs_written_on_the_call_s_stream_just_before():
    s = torch.cuda.Stream()
    q, k, v = rand(1, (2, 4, 64)), rand(2, (2, 2, 300, 64)), rand(3, (2, 2, 300, 64))
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    kk = torch.zeros_like(k)
    torch.cuda.synchronize()
    keep = _busy(s)
    with torch.cuda.stream(s):
        kk.copy_(k)
        lens.copy_(torch.tensor([300, 41], dtype=torch.int32, device="cuda"))
        o, lse = attn.decode_varlen(q, kk, v, lens)
    s.synchronize()
    del keep
    check_decode(o, lse, q, k, v, [300, 41], 0.0, None)


def test_captured_calls_follow_the_lengths_and_share_nothing():
    """Two graphs of decode steps, replayed at the same time on two streams
    while the lengths on the device grow, and a captured prefill."""
    B, Hq, Hkv, Ncap, D = 3, 8, 2, 400, 128
    sets = []
    for i in range(2):
        sets.append(dict(q=rand(i, (B, Hq, D)), k=rand(10 + i, (B, Hkv, Ncap, D)),
                         v=rand(20 + i, (B, Hkv, Ncap, D)), pk=rand(30 + i, (Hkv, 600, D)),
                         pv=rand(40 + i, (Hkv, 600, D)),
                         t=torch.zeros(B, dtype=torch.int32, device="cuda")))
    x = rand(60, (1, 2, 300, D))
    docs = torch.tensor([[100, 200]], dtype=torch.int32, device="cuda")
    attn.decode_varlen(sets[0]["q"], sets[0]["k"], sets[0]["v"], sets[0]["t"])
    torch.cuda.synchronize()
    graphs = []
    for i, c in enumerate(sets):
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c["a"] = attn.decode_varlen(c["q"], c["k"], c["v"], c["t"], softcap=30.0)
            c["b"] = attn.decode_prefix(c["q"], c["pk"], c["pv"], c["k"], c["v"], c["t"], softcap=30.0)
            if i == 0:
                c["f"] = attn.forward_mod(x, x, x, ranges=attn.row_ranges(docs, 300))
        graphs.append((g, s))
    for step in range(3):
        lens = [[step, 128 * step + 5, 399], [400, step + 1, 0]]
        for i, c in enumerate(sets):
            c["t"].copy_(torch.tensor(lens[i], dtype=torch.int32))
        docs.copy_(torch.tensor([[100 + step, 150]], dtype=torch.int32))
        torch.cuda.synchronize()
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for i, c in enumerate(sets):
            check_decode(*c["a"], c["q"], c["k"], c["v"], lens[i], 30.0, None)
            check_decode(*c["b"], c["q"], c["k"], c["v"], lens[i], 30.0, None, c["pk"], c["pv"])
        r = ranges_definition([[100 + step, 150]], None, 300, True).cuda()
        check_fwd(*sets[0]["f"], x, x, x, False, 1 / math.sqrt(D), 0.0, None, r, 0)


def test_helpers_refuse_wrong_tensors():
    q, k = rand(1, (1, 4, 16, 64)), rand(2, (1, 2, 16, 64))
    q1 = rand(1, (1, 4, 64))
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: attn.forward_mod(q.transpose(1, 2), k, k)),
        (ValueError, lambda: attn.forward_mod(q, k, k[:, :, :8].contiguous())),
        (ValueError, lambda: attn.forward_mod(q, k, k, slopes=torch.zeros(3, device="cuda"))),
        (TypeError, lambda: attn.forward_mod(q, k, k, slopes=torch.zeros(4, device="cuda").double())),
        (ValueError, lambda: attn.forward_mod(q, k, k, slopes=torch.zeros(4))),
        (ValueError, lambda: attn.forward_mod(q, k, k, ranges=torch.zeros(1, 15, 2, **i32))),
        (TypeError, lambda: attn.forward_mod(q, k, k, ranges=torch.zeros(1, 16, 2, device="cuda"))),
        (ValueError, lambda: attn.forward_mod(q, k, k, ranges=torch.zeros(1, 2, 16, **i32).transpose(1, 2))),
        (attn.AttnError, lambda: attn.forward_mod(q, k, k, q_offset=-1)),
        (attn.AttnError, lambda: attn.forward_mod(q, k, k, softcap=-1.0)),
        (ValueError, lambda: attn.decode_varlen(q1, k, k, torch.zeros(2, **i32))),
        (TypeError, lambda: attn.decode_varlen(q1, k, k, torch.zeros(1, device="cuda").long())),
        (ValueError, lambda: attn.decode_prefix(q1, k[0], k[0][:, :8].contiguous(), k, k)),
        (ValueError, lambda: attn.decode_prefix(q1, k[0, :1], k[0, :1], k, k)),
        (attn.AttnError, lambda: attn.row_ranges(torch.zeros(1, 2, **i32), 0)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()


def _guarded(shape, dtype, lead):
    """A buffer of one value around the tensor that is returned with it; the
    tensor starts `lead` bytes behind a 512-byte boundary."""
    size = math.prod(shape)
    each = torch.empty((), dtype=dtype).element_size()
    whole = torch.full((1024 + size + 1024,), 7.0, dtype=dtype, device="cuda")
    start = 512 + lead // each
    return whole, whole[start:start + size].view(shape), start


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lead", [0, 16])
def test_only_the_outputs_are_written(D, lead):
    """The C calls with outputs inside larger buffers, 32-byte aligned or only
    16-byte aligned: the same bits, and nothing around them changes."""
    B, Hq, Hkv, N = 2, 4, 2, 301
    x, kv = rand(1, (B, Hq, N, D)), rand(2, (B, Hkv, N, D))
    want = attn.forward_mod(x, kv, kv, causal=True, softcap=20.0)
    wo, o, at_o = _guarded((B, Hq, N, D), torch.bfloat16, lead)
    wl, lse, at_l = _guarded((B, Hq, N), torch.float32, lead)
    attn.attn_fwd_mod(x, kv, kv, o, lse, B, Hq, Hkv, N, N, D, 1, 0, D ** -0.5, 20.0)
    q, lens = x[:, :, 0].contiguous(), torch.tensor([301, 77], dtype=torch.int32, device="cuda")
    want_d = attn.decode_varlen(q, kv, kv, lens, softcap=20.0)
    wod, od, at_od = _guarded((B, Hq, D), torch.bfloat16, lead)
    wld, ld, at_ld = _guarded((B, Hq), torch.float32, lead)
    attn.attn_decode_varlen(q, kv, kv, lens, od, ld, B, Hq, Hkv, N, D, D ** -0.5, 20.0)
    wr, ranges, at_r = _guarded((B, N, 2), torch.int32, lead)
    docs = torch.tensor([[100, 150], [301, 0]], dtype=torch.int32, device="cuda")
    attn.attn_row_ranges(docs, None, ranges, B, N, 2, 1)
    torch.cuda.synchronize()
    assert torch.equal(ranges, attn.row_ranges(docs, N))
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(od, want_d[0]) and torch.equal(ld, want_d[1])
    for whole, out, at in ((wo, o, at_o), (wl, lse, at_l), (wod, od, at_od), (wld, ld, at_ld), (wr, ranges, at_r)):
        assert bool((whole[:at] == 7).all()) and bool((whole[at + out.numel():] == 7).all())


def test_the_same_call_gives_the_same_bits():
    """Whatever the order in which blocks run: prefill of ragged documents and
    decodes whose keys are cut in parts."""
    x = rand(1, (2, 8, 1500, 128))
    kv = rand(2, (2, 2, 1500, 128))
    r = attn.row_ranges(torch.tensor([[700, 20, 500], [3, 1400, 0]], dtype=torch.int32, device="cuda"), 1500)
    q = rand(3, (40, 8, 128))
    c = rand(4, (40, 2, 700, 128))
    p = rand(5, (2, 5000, 128))
    lens = torch.tensor([(37 * i) % 701 for i in range(40)], dtype=torch.int32, device="cuda")
    calls = (lambda: attn.forward_mod(x, kv, kv, ranges=r, softcap=30.0, slopes=alibi(8)),
             lambda: attn.decode_varlen(q, c, c, lens),
             lambda: attn.decode_prefix(q, p, p, c, c, lens, slopes=alibi(8)))
    for call in calls:
        first = call()
        for _ in range(5):
            again = call()
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_threads_with_streams_of_their_own_under_one_handle():
    """The per-thread default stream: one handle, another stream in each thread."""
    import threading
    per_thread = 2  # cudaStreamPerThread
    B, Hq, Hkv, Ncap, D = 4, 8, 2, 2000, 64
    lib, done = attn.load(), {}
    sets = []
    for i in range(3):
        lens = [1900 - 300 * i, 5 + i, 0, 777]
        sets.append((rand(i, (B, Hq, D)), rand(10 + i, (B, Hkv, Ncap, D)), rand(20 + i, (B, Hkv, Ncap, D)), lens,
                     torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     [(torch.empty((B, Hq, D), dtype=torch.bfloat16, device="cuda"),
                       torch.empty((B, Hq), device="cuda")) for _ in range(20)]))
    torch.cuda.synchronize()

    def work(i):
        q, k, v, _, t, outs = sets[i]
        torch.cuda.set_device(0)
        done[i] = [lib.attn_decode_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), t.data_ptr(), o.data_ptr(),
                                          lse.data_ptr(), B, Hq, Hkv, Ncap, D, 0.125, 0.0, None, per_thread)
                   for o, lse in outs]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, (q, k, v, lens, _, outs) in enumerate(sets):
        assert done[i] == [0] * 20
        for o, lse in outs:
            check_decode(o, lse, q, k, v, lens, 0.0, None)


def test_rows_of_more_keys_than_an_accumulator_takes():
    """128 rows of 1.9e8 keys, 128 that see the last key alone.  Every weight is 1 and
    every sum of one accumulator a multiple of 16 below 2^19: exact."""
    N = 190_000_000
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 49 GB")
    k = torch.zeros((1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.ones((1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
    ranges = torch.tensor([[[0, N]] * 128 + [[N - 1, N]] * 128], dtype=torch.int32, device="cuda")
    o, lse = attn.forward_mod(rand(1, (1, 1, 256, 64)), k, v, ranges=ranges)
    torch.cuda.synchronize()
    assert attn.attn_get_device_error() == 0
    assert bool((o == 1).all()) and bool((lse[..., 128:] == 0).all())
    assert bool(((lse[..., :128] - math.log(N)).abs() < 1e-4).all())


@pytest.mark.parametrize("heads", [2, 12])
def test_runs_of_more_keys_than_an_accumulator_takes(heads):
    """As above for single tokens: a CTA's share of the keys, own ones and those of a
    prefix, goes into several partial states."""
    N = 150_000_000
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 39 GB")
    k = torch.zeros((1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.ones((1, 1, N, 64), dtype=torch.bfloat16, device="cuda")
    q = rand(1, (1, heads, 64))
    lens = torch.tensor([N - 77], dtype=torch.int32, device="cuda")
    o, lse = attn.decode_varlen(q, k, v, lens)
    assert bool((o == 1).all()) and bool(((lse - math.log(N - 77)).abs() < 1e-4).all())
    own = k[:, :, :1000].contiguous()
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    o, lse = attn.decode_prefix(q, k[0], v[0], own, torch.ones_like(own), lens)
    assert bool((o == 1).all()) and bool(((lse - math.log(N + 1000)).abs() < 1e-4).all())


@pytest.mark.parametrize("D,cap,bias,kind", [
    (64, 0.0, 0, "causal"), (128, 20.0, 0, "ranges"), (64, 0.0, 1, "ranges"), (128, 20.0, -1, "causal ranges"),
    (64, 0.0, 0, "early")])
def test_prefill_of_several_segments_of_keys(D, cap, bias, kind):
    """Keys in three segments: rows that see all, some or none of them."""
    Hq, Hkv, Nq, Nk = 2, 1, 140, 600_000
    q, k, v = rand(1, (1, Hq, Nq, D)), rand(2, (1, Hkv, Nk, D)), rand(3, (1, Hkv, Nk, D))
    # (a bias of a few units over the length: both near and far keys count)
    slopes = torch.tensor([3e-6, 1e-5], device="cuda") * bias if bias else None
    q_offset = 1000 if kind == "early" else Nk - Nq - 30_000
    ranges = None
    if "ranges" in kind:
        rows = [(0, Nk), (5, 6), (262_143, 262_145), (262_144, 524_288), (300_000, 299_999), (100, 599_990),
                (524_200, Nk), (599_999, Nk + 50), (-3, 262_144)]
        ranges = torch.tensor([[rows[i % len(rows)] for i in range(Nq)]], dtype=torch.int32, device="cuda")
    causal = "causal" in kind or kind == "early"
    o, lse = attn.forward_mod(q, k, v, causal=causal, softcap=cap, slopes=slopes, ranges=ranges, q_offset=q_offset)
    check_fwd(o, lse, q, k, v, causal, 1 / math.sqrt(D), cap, slopes, ranges, q_offset)


@pytest.mark.parametrize("B,Hq,Hkv,Np,lens", [(1, 5, 1, 30_000, 700), (3, 4, 2, 9000, 9000), (150, 5, 1, 20_000, 90),
                                             (333, 5, 1, 20_000, 30), (401, 3, 1, 20_000, 30),
                                             (400, 8, 1, 20_000, 30)])
@pytest.mark.parametrize("D", [64, 128])
def test_few_and_many_rows_of_few_and_many_parts(B, Hq, Hkv, Np, lens, D):
    """Rows whose keys are cut in few or many parts, with any number of rows to a
    block of the merge."""
    own = [max(0, lens - 7 * i) for i in range(B)]
    q, k, v = rand(1, (B, Hq, D)), rand(2, (B, Hkv, lens, D)), rand(3, (B, Hkv, lens, D))
    pk, pv = rand(4, (Hkv, Np, D)), rand(5, (Hkv, Np, D))
    t = torch.tensor(own, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_prefix(q, pk, pv, k, v, t)
    some = sorted({0, 1 % B, B // 2, B - 1})
    check_decode(o, lse, q, k, v, own, 0.0, None, pk, pv, rows=some)
    o, lse = attn.decode_varlen(q, k, v, t)
    check_decode(o, lse, q, k, v, own, 0.0, None, rows=some)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [50.0, 200.0, 1000.0])
@pytest.mark.parametrize("causal", [False, True])
def test_capped_rows_behind_tiles_that_they_do_not_see(D, cap, causal):
    """Rows of a second document, all of whose scores are far below 0, among 16 rows
    whose others see tiles in front of it: what those tiles hold has no say in them."""
    N, first = 600, 200  # rows 192 .. 199 are the first document's, 200 .. 207 not
    q = (1 + 0.1 * rand(1, (1, 2, N, D)).float()).bfloat16()
    k = 0.1 * rand(2, (1, 2, N, D)).float()
    k[:, :, first:] -= 150 * D ** -0.5  # scores about -150
    k, v = k.bfloat16(), rand(3, (1, 2, N, D))
    ranges = attn.row_ranges(torch.tensor([[first, N - first]], dtype=torch.int32, device="cuda"), N, causal=causal)
    o, lse = attn.forward_mod(q, k, v, softcap=cap, ranges=ranges)
    check_fwd(o, lse, q, k, v, False, D ** -0.5, cap, None, ranges, 0)


def _calls_on(stream):
    """Each helper on `stream`: (call, output shapes and types)."""
    q, k = rand(1, (2, 4, 1500, 64)), rand(2, (2, 2, 1500, 64))
    q1, p = rand(3, (2, 4, 64)), rand(4, (2, 900, 64))
    lens = torch.tensor([1500, 700], dtype=torch.int32, device="cuda")
    docs = torch.tensor([[1000, 300], [20, 1]], dtype=torch.int32, device="cuda")
    return [lambda: attn.forward_mod(q, k, k, causal=True, stream=stream),
            lambda: attn.decode_varlen(q1, k, k, lens, stream=stream),
            lambda: attn.decode_prefix(q1, p, p, k, k, lens, stream=stream),
            lambda: (attn.row_ranges(docs, 1500, stream=stream),)]


@pytest.mark.parametrize("which", range(4), ids=["forward_mod", "decode_varlen", "decode_prefix", "row_ranges"])
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_on_another_stream_take_no_memory_that_is_still_read(which, handle):
    """Freed memory that the current stream is still to read is not written by a call on
    another stream; nor are that call's outputs by the next one, once they are freed,
    while the current stream is still to read them."""
    side = torch.cuda.Stream()
    call = _calls_on(side.cuda_stream if handle else side)[which]
    want = [x.clone() for x in _calls_on(None)[which]()]
    torch.cuda.synchronize()
    # memory of the outputs' sizes, read by the current stream long after it is freed
    olds = [torch.full_like(x, 3) for _ in range(4) for x in want]
    torch.cuda.synchronize()
    busy = _busy(torch.cuda.current_stream())
    reads = [x.clone() for x in olds]
    del olds
    for _ in range(4):
        got = call()
    side.synchronize()  # (the current stream is still busy)
    torch.cuda.synchronize()
    assert all(bool((x == 3).all()) for x in reads)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # the outputs themselves, read by the current stream after they are freed
    got = call()
    torch.cuda.current_stream().wait_stream(side)
    del busy
    busy = _busy(torch.cuda.current_stream())
    reads = [x.clone() for x in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full_like(x, 5) for _ in range(4) for x in want]
    torch.cuda.synchronize()
    del busy, over
    assert all(torch.equal(x, y) for x, y in zip(reads, want))


def test_helpers_refuse_values_that_change_on_their_way_to_c():
    q, docs = rand(1, (1, 2, 16, 64)), torch.tensor([[10, 6]], dtype=torch.int32, device="cuda")
    for call in (lambda: attn.forward_mod(q, q, q, causal=True, q_offset=2**32),
                 lambda: attn.forward_mod(q, q, q, causal=True, q_offset=5 - 2**32),
                 lambda: attn.row_ranges(docs, 2**32 + 16), lambda: attn.row_ranges(docs, 16 - 2**32),
                 lambda: attn.forward_mod(q, q, q, softcap=1e-46),
                 lambda: attn.decode_varlen(q[:, :, 0].contiguous(), q, q, softcap=1e-46)):
        with pytest.raises(attn.AttnError):
            call()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (12.0, False), (0.0, True), (12.0, True)],
                         ids=["plain", "cap", "bias", "both"])
@pytest.mark.parametrize("kind", ["all", "causal", "ranges", "causal ranges"])
def test_items_one_after_another_on_a_cta(D, cap, bias, kind):
    """More work items than CTAs, every row checked: what an item leaves behind (Q, the
    rows' data, the parities of every barrier) is not what the next one takes.  With
    ranges the items are of very different lengths, some of them empty."""
    B, Hq, Hkv, Nq, Nk = 3, 24, 12, 1100, 1300
    q, k, v = rand(1, (B, Hq, Nq, D), 3.0), rand(2, (B, Hkv, Nk, D)), rand(3, (B, Hkv, Nk, D))
    slopes = alibi(Hq) if bias else None
    ranges = None
    if "ranges" in kind:
        lens = torch.tensor([[1, 300, 2, 500, 97, 130], [0, 0, 600, 0, 0, 0], [7, 7, 400, 600, 0, 0]],
                            dtype=torch.int32, device="cuda")
        ranges = attn.row_ranges(lens, Nq, causal=False)
    causal, q_offset = "causal" in kind, 77
    o, lse = attn.forward_mod(q, k, v, causal=causal, q_offset=q_offset, softcap=cap, slopes=slopes, ranges=ranges)
    check_fwd(o, lse, q, k, v, causal, D ** -0.5, cap, slopes, ranges, q_offset)


def _sizes(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


@pytest.mark.parametrize("seed", range(24))
def test_random_prefills(seed):
    import random
    rng = random.Random(1000 + seed)
    D, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 3]), rng.choice([1, 2, 4, 5])
    B, Nq, Nk = rng.randint(1, 3), _sizes(rng, 1, 700), _sizes(rng, 1, 900)
    Hq, causal, q_offset = Hkv * G, rng.random() < 0.5, rng.choice([0, 0, rng.randint(0, 900)])
    cap, sigma = rng.choice([0.0, 0.7, 20.0, 50.0, 300.0]), rng.choice([0.1, 1.0, 8.0, 40.0])
    kind = rng.choice([None, "wild", "narrow", "docs", "prefix", "none"])
    if kind in ("docs", "prefix") and Nq < 8:
        kind = "wild"
    slopes = None
    if rng.random() < 0.5:
        slopes = torch.tensor([rng.choice([1, 1, -1, 0]) * 10 ** rng.uniform(-4, 1) for _ in range(Hq)],
                              dtype=torch.float32, device="cuda")
    q, k, v = rand(seed, (B, Hq, Nq, D), sigma), rand(seed + 100, (B, Hkv, Nk, D)), rand(seed + 200, (B, Hkv, Nk, D))
    # scores of one sign in parts, so that a row's keys differ from its neighbours'
    if rng.random() < 0.5:
        q += sigma
        k[:, :, Nk // 2:] -= 1
    ranges = ranges_of(kind, B, Nq, Nk, seed)
    scale = rng.choice([D ** -0.5, 0.02, 1.0])
    o, lse = attn.forward_mod(q, k, v, causal=causal, q_offset=q_offset, softcap=cap, slopes=slopes, ranges=ranges,
                              scale=scale)
    check_fwd(o, lse, q, k, v, causal, scale, cap, slopes, ranges, q_offset, f"{D, B, Hq, Hkv, Nq, Nk, cap, kind}")


@pytest.mark.parametrize("seed", range(24))
def test_random_decodes(seed):
    import random
    rng = random.Random(2000 + seed)
    D, Hkv, G = rng.choice([64, 128]), rng.choice([1, 2, 3]), rng.choice([1, 2, 4, 5, 8, 9, 16, 33])
    B, Ncap, Np = _sizes(rng, 1, 60), _sizes(rng, 1, 2000), _sizes(rng, 1, 9000)
    Hq, cap, sigma = Hkv * G, rng.choice([0.0, 0.7, 20.0, 300.0]), rng.choice([0.1, 1.0, 8.0])
    lens = [rng.choice([0, 1, Ncap, rng.randint(0, Ncap)]) for _ in range(B)]
    slopes = None
    if rng.random() < 0.5:
        slopes = torch.tensor([rng.choice([1, 1, -1, 0]) * 10 ** rng.uniform(-4, 0) for _ in range(Hq)],
                              dtype=torch.float32, device="cuda")
    q, k, v = rand(seed, (B, Hq, D), sigma), rand(seed + 100, (B, Hkv, Ncap, D)), rand(seed + 200, (B, Hkv, Ncap, D))
    pk, pv = rand(seed + 300, (Hkv, Np, D)), rand(seed + 400, (Hkv, Np, D))
    for b, n in enumerate(lens):
        for x in (k, v):
            x[b, :, n:] = (NAN, INF, -INF)[b % 3]
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    some = sorted({0, B - 1, *(rng.randrange(B) for _ in range(4))})
    o, lse = attn.decode_varlen(q, k, v, t, softcap=cap, slopes=slopes)
    check_decode(o, lse, q, k, v, lens, cap, slopes, rows=some)
    o, lse = attn.decode_prefix(q, pk, pv, k, v, t, softcap=cap, slopes=slopes)
    check_decode(o, lse, q, k, v, lens, cap, slopes, pk, pv, rows=some)


@pytest.mark.parametrize("D", [64, 128])
def test_query_and_output_offsets_beyond_32_bits(D):
    """More than 2^32 elements of Q and O: the last rows of the last heads are theirs."""
    if torch.cuda.mem_get_info()[0] < 60 * 2**30:
        pytest.skip("needs 40 GB")
    Hq, Hkv, Nk, tail = 64, 2, 5000, 300
    Nq = 2**32 // (Hq * D) + 1111
    q = torch.zeros((1, Hq, Nq, D), dtype=torch.bfloat16, device="cuda")
    heads = (0, Hq // 2 - 1, Hq - 1)
    for h in heads:
        q[0, h, Nq - tail:] = rand(h, (tail, D))
    k, v = rand(100, (1, Hkv, Nk, D)), rand(101, (1, Hkv, Nk, D))
    lo = (torch.arange(Nq, device="cuda") * (Nk - 50) // Nq).int()
    ranges = torch.stack([lo, lo + 50], -1)[None].contiguous()
    o, lse = attn.forward_mod(q, k, v, ranges=ranges, softcap=20.0)
    j, rows = torch.arange(Nk, device="cuda"), slice(Nq - tail, Nq)
    seen = (j >= ranges[0, rows, :1]) & (j < ranges[0, rows, 1:])
    for h in heads:
        ref = definition(q[0, h, rows], k[0, h // 32], v[0, h // 32], j[:tail], j, seen, D ** -0.5, 20.0, None)
        check(o[0, h, rows], lse[0, h, rows], ref, f"h{h}")


def test_captured_prefill_of_several_segments_beside_an_eager_one():
    """The accumulators of segments belong to their call: two graphs and an eager call at
    once, each replayed on keys that changed."""
    Hq, Nq, Nk, D = 2, 130, 300_000, 64
    sets, graphs = [], []
    for i in range(3):
        sets.append([rand(i, (1, Hq, Nq, D)), rand(10 + i, (1, 1, Nk, D)), rand(20 + i, (1, 1, Nk, D))])
    torch.cuda.synchronize()
    for q, k, v in sets[:2]:
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            out = attn.forward_mod(q, k, v, softcap=30.0)
        graphs.append((g, s, out))
    for turn in range(2):
        for i, x in enumerate(sets):
            x[1].copy_(rand(50 + 3 * turn + i, x[1].shape))
        torch.cuda.synchronize()
        for g, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager = attn.forward_mod(*sets[2], softcap=30.0)
        torch.cuda.synchronize()
        for x, out in zip(sets, [graphs[0][2], graphs[1][2], eager]):
            check_fwd(*out, *x, False, 1 / 8, 30.0, None, None, 0)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (24, 2)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_nan_in_a_query_or_a_request_s_keys_stays_there(Hq, Hkv, cap, bias):
    lens = [300, 40, 129, 0]
    q, k, v = rand(1, (4, Hq, 64)), rand(2, (4, Hkv, 300, 64)), rand(3, (4, Hkv, 300, 64))
    pk, pv = rand(4, (Hkv, 1000, 64)), rand(5, (Hkv, 1000, 64))
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slopes = alibi(Hq) if bias else None
    clean = [attn.decode_varlen(q, k, v, t, softcap=cap, slopes=slopes),
             attn.decode_prefix(q, pk, pv, k, v, t, softcap=cap, slopes=slopes)]
    q[0, 3], k[1, 1, 17], k[2, 0, 128, 5] = NAN, NAN, NAN
    G = Hq // Hkv
    hit = torch.zeros(4, Hq, dtype=torch.bool, device="cuda")
    hit[0, 3], hit[1, G:], hit[2, :G] = True, True, True
    dirty = [attn.decode_varlen(q, k, v, t, softcap=cap, slopes=slopes),
             attn.decode_prefix(q, pk, pv, k, v, t, softcap=cap, slopes=slopes)]
    for (o, lse), (co, cl) in zip(dirty, clean):
        assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
        # (a running maximum that a NaN keeps in place is another reference: not other values)
        assert torch.equal(torch.isinf(lse[~hit]), torch.isinf(cl[~hit]))
        assert torch.allclose(o[~hit].float(), co[~hit].float(), atol=2.0**-6, rtol=2.0**-7)
        fin = ~torch.isinf(cl) & ~hit
        assert torch.allclose(lse[fin], cl[fin], atol=1e-4, rtol=0)


def test_calls_captured_on_a_stream_beside_the_capturing_one():
    q, k, v = rand(1, (3, 8, 64)), rand(2, (3, 2, 500, 64)), rand(3, (3, 2, 500, 64))
    x, lens = rand(4, (1, 2, 300, 64)), torch.tensor([500, 3, 77], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g, s, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        side.wait_stream(s)
        a = attn.decode_varlen(q, k, v, lens, stream=side)
        b = attn.forward_mod(x, x, x, causal=True, stream=side)
        c = attn.decode_varlen(q, k, v, lens, softcap=5.0)
        s.wait_stream(side)
        d = attn.forward_mod(x, x, x, softcap=5.0)
    for turn in range(2):
        lens.copy_(torch.tensor([400 + turn, 0, 78], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check_decode(*a, q, k, v, [400 + turn, 0, 78], 0.0, None)
        check_decode(*c, q, k, v, [400 + turn, 0, 78], 5.0, None)
        check_fwd(*b, x, x, x, True, 1 / 8, 0.0, None, None, 0)
        check_fwd(*d, x, x, x, False, 1 / 8, 5.0, None, None, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slope", [4.0, 4.7, 17.0, 100.0, 3e4])
@pytest.mark.parametrize("cap", [0.0, 20.0, 100.0])
def test_steep_biases(D, slope, cap):
    """Slopes at which a few keys, or one, have all the weight: the roundings of biases
    of keys far from those have no part in the result."""
    q, k, v = rand(1, (1, 4, 300, D), 0.05), rand(2, (1, 2, 400, D)), rand(3, (1, 2, 400, D))
    slopes = torch.tensor([slope, -slope, slope / 3, 0.1], device="cuda")
    i = torch.arange(300, device="cuda")
    one = torch.stack([i + 50, i + 51], -1)[None].int()  # each row sees the key at its position alone
    for causal, kind in ((True, None), (False, "prefix"), (False, "narrow"), (False, "one"), (False, "before")):
        ranges = one if kind == "one" else one - 30 if kind == "before" else ranges_of(kind, 1, 300, 400)
        o, lse = attn.forward_mod(q, k, v, causal=causal, q_offset=50, softcap=cap, slopes=slopes, ranges=ranges)
        check_fwd(o, lse, q, k, v, causal, D ** -0.5, cap, slopes, ranges, 50, kind)
    q1, pk, pv = rand(4, (3, 4, D), 0.05), rand(5, (2, 333, D)), rand(6, (2, 333, D))
    k3, v3 = rand(7, (3, 2, 200, D)), rand(8, (3, 2, 200, D))
    lens = [200, 0, 17]
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = attn.decode_prefix(q1, pk, pv, k3, v3, t, softcap=cap, slopes=slopes)
    check_decode(o, lse, q1, k3, v3, lens, cap, slopes, pk, pv)
    o, lse = attn.decode_varlen(q1, k3, v3, t, softcap=cap, slopes=slopes)
    check_decode(o, lse, q1, k3, v3, lens, cap, slopes)
