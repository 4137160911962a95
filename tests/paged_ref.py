"""Paged caches and their operators by definition, in 64 bits: what tests/test_gpu_paged.py
compares with.  Everything but the inputs is made by loops over requests and heads."""
import math

import torch

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def decode_e4m3(code):
    """Value of an e4m3 code (a Python int), from the format: 1 sign, 4 exponent, 3 mantissa
    bits, bias 7, subnormals m / 8 * 2^-6."""
    s, e, m = code >> 7, code >> 3 & 15, code & 7
    x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
    return -x if s else x


E4M3_VALUES = torch.tensor([decode_e4m3(c) for c in range(256)], dtype=torch.float64)


def quantise(x):
    """(codes as values / 2^e in 64 bits, e) of the rows of x [..., D], by the definition."""
    x = x.double()
    a = x.abs().amax(-1)
    e = torch.full(a.shape, -100, dtype=torch.int64, device=x.device)
    for k in range(-100, 100):  # the least e in [-100, 100] with a <= 448 2^e
        e = torch.where(a > 448 * 2.0 ** k, torch.full_like(e, k + 1), e)
    e = torch.where(a == 0, torch.zeros_like(e), e)
    y = (x * torch.exp2(-e.double()).unsqueeze(-1)).clamp(-448, 448)
    exponent = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(y / step) * step, e


class Cache:
    """Pages dealt out to B requests in an order of the seed.  Slots that hold no token hold
    NaN (bf16), or the codes and scale byte of NaN (quantised); entries of the table behind a
    request's last page are out of range."""

    def __init__(self, lens, Hkv, D, page, quant, seed=0, spare=3, sigma=1.0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.page, self.quant = list(lens), Hkv, D, page, quant
        B = len(lens)
        pages = [-(-n // page) for n in lens]
        P, M = sum(pages) + spare, max(1, max(pages))
        ids = torch.randperm(P, generator=g).tolist()
        table = torch.full((B, M), 2**31 - 1, dtype=torch.int32)
        for b in range(B):
            for i in range(pages[b]):
                table[b, i] = ids.pop()
        self.table = table.to(device)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.dense = []  # per request (k, v) [n, Hkv, D] in 64 bits, as the cache holds them
        kv = []
        for n in lens:
            kv.append([(torch.randn(n, Hkv, D, generator=g) * sigma).to(BF16).to(device) for _ in range(2)])
        shape = (P, Hkv, page, D)
        if quant:
            self.kp, self.vp = (torch.full(shape, 0x7F, dtype=torch.uint8, device=device).view(E4M3)
                                for _ in range(2))
            self.ks, self.vs = (torch.full(shape[:3], 255, dtype=torch.uint8, device=device) for _ in range(2))
        else:
            self.kp, self.vp = (torch.full(shape, float("nan"), dtype=BF16, device=device) for _ in range(2))
            self.ks = self.vs = None
        for b, n in enumerate(lens):
            both = []
            for x, pages_, scale in zip(kv[b], (self.kp, self.vp), (self.ks, self.vs)):
                if quant:
                    y, e = quantise(x)
                    both.append(y * torch.exp2(e.double()).unsqueeze(-1))
                    x = y.to(torch.float32).to(E4M3)
                for i in range(pages[b]):
                    m = min(page, n - i * page)
                    rows = slice(i * page, i * page + m)
                    at = int(table[b, i])
                    if quant:
                        pages_.view(torch.uint8)[at, :, :m] = x.view(torch.uint8)[rows].transpose(0, 1)
                        scale[at, :, :m] = (e[rows] + 127).to(torch.uint8).transpose(0, 1)
                    else:
                        pages_[at, :, :m] = x[rows].transpose(0, 1)
                if not quant:
                    both.append(x.double())
            self.dense.append(both)

    def args(self):
        return self.kp, self.vp, self.table, self.lens_t

    def scales(self):
        return dict(kscale=self.ks, vscale=self.vs) if self.quant else {}


def offsets_of(new, device="cuda", first=0):
    out = [first]
    for n in new:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


def attend(q, cache, offsets, scale, causal=True):
    """(o, lse, spread) in 64 bits of q [T, Hq, D]; spread = sum_j softmax_j |v_j|, what a
    relative error of the weights is multiplied by.  Rows of no request: NaN."""
    T, Hq, D = q.shape
    G = Hq // cache.Hkv
    o, spread = (torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64, device=q.device)
    off = offsets.tolist()
    for b, (k, v) in enumerate(cache.dense):
        n, m = off[b + 1] - off[b], cache.lens[b]
        rows = slice(off[b], off[b + 1])
        if n == 0:
            continue
        pos = torch.arange(n, device=q.device) + (m - n)
        seen = torch.arange(m, device=q.device)[None, :] <= (pos[:, None] if causal else m)
        for h in range(Hq):
            x = scale * (q[rows, h].double() @ k[:, h // G].T)
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(1, keepdim=True) if m else torch.full((n, 1), -math.inf, device=q.device)
            none = torch.isinf(top)
            w = torch.where(none, torch.zeros_like(x), torch.exp(x - top))
            total = w.sum(1, keepdim=True)
            w = w / torch.where(none, torch.ones_like(total), total)
            o[rows, h], spread[rows, h] = w @ v[:, h // G], w @ v[:, h // G].abs()
            lse[rows, h] = torch.where(none, top, top + torch.log(total)).squeeze(1)
    return o, lse, spread
