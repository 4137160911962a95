"""Cases of the paged key/value cache and the attention that reads it, and their plain forms.

Four operators of ``attention_forward_sm_gb300`` over a cache of pages, each holding ``page`` tokens
of every KV head; ``table[b]`` names the pages of request b in order:

* ``write``   ``cache_write``: puts new tokens' K and V into their pages, as bf16 or quantised to
  e4m3 with a power-of-two scale for each token and KV head;
* ``read``    ``cache_read``: the last tokens of each request as dense bf16 rows;
* ``decode``  ``paged_decode``: one new token per request against its cache;
* ``chunk``   ``paged_forward``: several new tokens per request (a chunk of a prompt, a few
  drafted tokens to verify, both in one batch), each seeing the tokens up to itself.

Definitions.  Request b has lens[b] tokens in its cache, the last n_b of them new; its new tokens
are the rows offsets[b] .. offsets[b+1] of q, k and v, row i at position p = lens[b] - n_b + i,
which is slot p % page of page table[b][p // page].

Attention: O = sum_j softmax(scale q.k_j) v_j and LSE = ln sum_j exp(scale q.k_j) over the keys
j <= p (none: 0 and -inf).

Quantised: a row x of D values with largest magnitude a has the scale 2^e, e the least integer with
a <= 448 * 2^e (0 for a row of zeros; at least -100, at most 100), stored as the byte e + 127, and
the codes e4m3(x / 2^e), rounded to nearest, ties to even.  Read back it is code * 2^e, which bf16
holds exactly.
"""
import math

import torch

own = False


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # the smallest call: the token that each of a few requests has just produced
        dict(name="write tokens", op="write", B=8, Hkv=8, D=128, page=16, quant=False,
             ctx_lo=100, ctx_hi=1000, new_lo=1, new_hi=1),
        # prompts of very different lengths, quantised on their way into the cache
        dict(name="write prompts e4m3", op="write", B=24, Hkv=8, D=128, page=64, quant=True,
             ctx_lo=1, ctx_hi=1, new_lo=100, new_hi=4001),
        # short contexts of a small model handed on to another step, odd lengths, the smallest pages
        dict(name="read odd", op="read", B=5, Hkv=3, D=64, page=16, quant=False,
             ctx_lo=1, ctx_hi=1, new_lo=33, new_hi=2011),
        # long contexts out of a quantised cache
        dict(name="read long e4m3", op="read", B=8, Hkv=8, D=128, page=64, quant=True,
             ctx_lo=1, ctx_hi=1, new_lo=2000, new_hi=60000),
        # one request with a short context: the latency of a decode step
        dict(name="decode one", op="decode", B=1, Hkv=8, G=4, D=128, page=16, quant=False,
             ctx_lo=1022, ctx_hi=1022, new_lo=1, new_hi=1),
        # a batch whose requests are of very different lengths
        dict(name="decode ragged 64k", op="decode", B=8, Hkv=8, G=4, D=128, page=64, quant=False,
             ctx_lo=500, ctx_hi=65535, new_lo=1, new_hi=1),
        # a serving batch over a quantised cache
        dict(name="decode serving e4m3", op="decode", B=64, Hkv=8, G=8, D=128, page=32, quant=True,
             ctx_lo=16, ctx_hi=12000, new_lo=1, new_hi=1),
        # drafted tokens to verify: a few rows for each request
        dict(name="chunk verify", op="chunk", B=16, Hkv=8, G=4, D=128, page=16, quant=False,
             ctx_lo=100, ctx_hi=16384, new_lo=4, new_hi=4),
        # a chunk of one long prompt
        dict(name="chunk prompt", op="chunk", B=1, Hkv=8, G=4, D=128, page=128, quant=False,
             ctx_lo=16001, ctx_hi=16001, new_lo=2048, new_hi=2048),
        # the same over a quantised cache, a smaller chunk behind a longer context
        dict(name="chunk prompt e4m3", op="chunk", B=1, Hkv=8, G=4, D=128, page=64, quant=True,
             ctx_lo=30000, ctx_hi=30000, new_lo=1024, new_hi=1024),
        # prompts' chunks and single tokens in one batch
        dict(name="chunk mixed e4m3", op="chunk", B=12, Hkv=4, G=4, D=128, page=32, quant=True,
             ctx_lo=64, ctx_hi=6000, new_lo=1, new_hi=500),
        # odd everything: seven query heads to a KV head, the small head size
        dict(name="chunk odd", op="chunk", B=3, Hkv=2, G=7, D=64, page=16, quant=False,
             ctx_lo=5, ctx_hi=4099, new_lo=77, new_hi=700),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "chunk", "chunk", "chunk"])
    c = dict(op=op, Hkv=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128]), quant=rng.random() < 0.5)
    if op in ("write", "read"):
        # up to as many tokens in all as the largest listed read
        c["B"] = _log_int(rng, 1, 64)
        most = _log_int(rng, 1, 120000 // c["B"])
        least = _log_int(rng, 1, most)
        c.update(ctx_lo=1, ctx_hi=_log_int(rng, 1, max(1, 20000 // c["B"])), new_lo=least, new_hi=most)
        return c
    c["G"] = rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
    if op == "decode":
        longest = _log_int(rng, 100, 65536)
        c["B"] = _log_int(rng, 1, max(1, min(128, 500000 // longest)))
        c.update(ctx_lo=_log_int(rng, 1, longest), ctx_hi=longest, new_lo=1, new_hi=1)
        return c
    heads = c["Hkv"] * c["G"]
    longest = _log_int(rng, 64, 32768)
    # no more scores than the largest listed case, were every request as long as the longest
    scores = 32 * 2048 * 17025
    most = _log_int(rng, 1, max(1, min(2048, scores // (heads * longest))))
    c["B"] = _log_int(rng, 1, max(1, min(32, scores // (heads * longest * most), 500000 // longest)))
    c.update(ctx_lo=_log_int(rng, 1, longest), ctx_hi=longest, new_lo=_log_int(rng, 1, most), new_hi=most)
    return c


# ----------------------------------------------------------------------------- lengths


def _quantiles(lo, hi, n):
    """n whole numbers: quantiles of a log-uniform distribution on [lo, hi]."""
    if n == 1:
        return [hi]
    return [max(lo, min(hi, round(lo * (hi / lo) ** (i / (n - 1))))) for i in range(n)]


def _lengths(case):
    """(new tokens, tokens in the cache) of every request.  Which context goes with which number
    of new tokens is fixed (a third of the way round), so that every seed has the same work."""
    B = case["B"]
    new, ctx = (_quantiles(case[x + "_lo"], case[x + "_hi"], B) for x in ("new", "ctx"))
    # the shortest context of a written or read request is none at all
    ctx = [0 if c == 1 and case["op"] in ("write", "read") else c for c in ctx]
    return [(new[i], new[i] + ctx[(i + B // 3) % B]) for i in range(B)]


def work(case):
    op, Hkv, D = case["op"], case["Hkv"], case["D"]
    lengths = _lengths(case)
    row = Hkv * (D + 1 if case["quant"] else 2 * D)  # a token's K or V in the cache
    tokens, keys = sum(n for n, _ in lengths), sum(m for _, m in lengths)
    pages = 4 * sum(-(-m // case["page"]) for _, m in lengths)
    if op in ("write", "read"):
        touched = 4 * sum(-(-n // case["page"]) for n, _ in lengths)
        return {"bytes": 2 * tokens * (row + 2 * Hkv * D) + touched + 8 * case["B"],
                "flops": 4 * tokens * Hkv * D if case["quant"] else 0}
    Hq = Hkv * case["G"]
    pairs = sum(n * m - n * (n - 1) // 2 for n, m in lengths)
    return {"bytes": 2 * keys * row + tokens * Hq * (4 * D + 4) + pages + 8 * case["B"], "flops": 4 * D * Hq * pairs}


# ----------------------------------------------------------------------------- inputs


def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """Codes and scale bytes of the rows of x [..., D]."""
    x = x.float()
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, 1/2 <= m < 1, and 448 = 7/8 2^9
    e = torch.where(a > 0, (e - 9 + (m > 0.875).int()).clamp(-100, 100), 0)
    codes = (x * _pow2(-e).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _normal(gen, shape):
    return torch.randn(shape, generator=gen, dtype=torch.float32, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * int(seed) + 29)
    s = dict(case)
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    Hq = Hkv * case.get("G", 0)
    order = torch.randperm(B, generator=gen, device="cuda").tolist()
    lengths = [_lengths(case)[i] for i in order]
    new, lens = [n for n, _ in lengths], [m for _, m in lengths]
    pages = [-(-m // page) for m in lens]
    # a pool with some pages to spare, dealt out in any order; -1 behind a request's last page
    P = sum(pages) + 7
    ids = torch.randperm(P, generator=gen, device="cuda").to(torch.int32).tolist()
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = torch.tensor(ids[at:at + pages[b]], dtype=torch.int32)
        at += pages[b]
    s["table"] = table.cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["offsets"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["rows"], s["max_new"] = sum(new), max(new)
    s["kscale"] = s["vscale"] = None
    if case["op"] == "write":  # K and V behind a projection that makes both, and an empty cache
        kv = _normal(gen, (s["rows"], 2 * Hkv, D))
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        kind = torch.float8_e4m3fn if case["quant"] else torch.bfloat16
        s["kp"], s["vp"] = (torch.zeros(P, Hkv, page, D, dtype=torch.bfloat16, device="cuda").to(kind)
                            for _ in range(2))
        if case["quant"]:
            s["kscale"], s["vscale"] = (torch.full((P, Hkv, page), 127, dtype=torch.uint8, device="cuda")
                                        for _ in range(2))
        return s
    s["kp"], s["vp"] = _normal(gen, (P, Hkv, page, D)), _normal(gen, (P, Hkv, page, D))
    if case["quant"]:
        s["kp"], s["kscale"] = _quantise(s["kp"])
        s["vp"], s["vscale"] = _quantise(s["vp"])
    if Hq:  # the queries, out of a projection that makes q, k and v
        s["q"] = _normal(gen, (s["rows"], Hq + 2 * Hkv, D))[:, :Hq]
    return s


# ----------------------------------------------------------------------------- plain forms


def _places(s):
    """(page, slot) of every new token, in the order of the rows."""
    off = s["offsets"].long()
    i = torch.arange(s["rows"], device=off.device)
    b = torch.searchsorted(off, i, right=True) - 1
    pos = s["lens"].long()[b] - off[b + 1] + i
    return s["table"].long()[b, pos // s["page"]], pos % s["page"]


def _bytes(x):
    return x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x


def _plain_write(s):
    page, slot = _places(s)
    out = []
    for x, pages, scale in ((s["k"], s["kp"], s["kscale"]), (s["v"], s["vp"], s["vscale"])):
        if scale is not None:
            x, e = _quantise(x)
            scale[page, :, slot] = e
            out.append(scale)
        _bytes(pages)[page, :, slot] = _bytes(x)
        out.append(pages)
    return out


def _values(pages, scale, index):
    """fp32 values of the rows pages[index] (index: a tuple of tensors and slices)."""
    x = _bytes(pages)[index].view(pages.dtype).float()
    return x if scale is None else x * _pow2(scale[index].int() - 127).unsqueeze(-1)


def _plain_read(s):
    page, slot = _places(s)
    at = (page, slice(None), slot)
    return [_values(s["kp"], s["kscale"], at).to(torch.bfloat16), _values(s["vp"], s["vscale"], at).to(torch.bfloat16)]


def _plain_attend(s):
    """Every request padded to the longest context and to the most new tokens."""
    B, Hkv, G, D, page = s["B"], s["Hkv"], s["G"], s["D"], s["page"]
    Hq, N = Hkv * G, s["max_new"]
    table, lens, off = s["table"].long().clamp(min=0), s["lens"].long(), s["offsets"].long()
    n = table.shape[1] * page
    k, v = (_values(x, e, (table,)).transpose(1, 2).reshape(B, Hkv, n, D)
            for x, e in ((s["kp"], s["kscale"]), (s["vp"], s["vscale"])))
    i = torch.arange(N, device=lens.device)
    new = off[1:] - off[:-1]
    real = i < new[:, None]  # [B, N]: rows that there are
    q = s["q"][(off[:-1, None] + i).clamp(max=s["rows"] - 1)].float()  # [B, N, Hq, D]
    q = q.view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(D)).view(B, Hkv, N, G, n)
    last = lens[:, None] - new[:, None] + i  # [B, N]
    unseen = torch.arange(n, device=lens.device) > last[..., None]  # [B, N, n]
    x.masked_fill_(unseen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, N * G, n), v).view(B, Hkv, N, G, D) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(-1)  # [B, Hkv, N, G]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)[real]
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(B, N, Hq)[real]


def run(state):
    s = state
    op = s["op"]
    if own:
        import attention_forward_sm_gb300 as attn
        cache = (s["kp"], s["vp"], s["table"], s["lens"])
        scales = dict(kscale=s["kscale"], vscale=s["vscale"])
        if op == "write":
            attn.cache_write(s["k"], s["v"], *cache, s["offsets"], **scales)
            return ([s["kscale"], s["kp"], s["vscale"], s["vp"]] if s["quant"] else [s["kp"], s["vp"]])
        if op == "read":
            return list(attn.cache_read(*cache, s["offsets"], s["rows"], **scales))
        if op == "decode":
            return attn.paged_decode(s["q"], *cache, **scales)
        return attn.paged_forward(s["q"], *cache, s["offsets"], max_new=s["max_new"], **scales)
    if op == "write":
        return _plain_write(s)
    return _plain_read(s) if op == "read" else _plain_attend(s)


# ----------------------------------------------------------------------------- 64 bits


def _exact_codes(x):
    """e4m3 of the rows of x [..., D] as numbers in 64 bits, by the definition: 4 significant
    bits, steps of 2^-9 at the least, ties to the even step."""
    x = x.double()
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(a / 448))
    # (log2 may be off where a / 448 is next to a power of two)
    e = torch.where(a <= 448 * torch.exp2(e - 1), e - 1, torch.where(a > 448 * torch.exp2(e), e + 1, e))
    e = torch.where(a > 0, e.clamp(-100, 100), torch.zeros_like(e))
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hkv, D, page = case["op"], case["B"], case["Hkv"], case["D"], case["page"]
    off, lens, table = s["offsets"].tolist(), s["lens"].tolist(), s["table"].tolist()
    if op == "write":
        if not case["quant"]:
            return None  # copies
        out = []
        for x, pages in ((s["k"], s["kp"]), (s["v"], s["vp"])):
            y, codes = torch.zeros(pages.shape, dtype=torch.float64, device="cuda"), _exact_codes(x)
            for b in range(B):
                n = off[b + 1] - off[b]
                done = 0
                while done < n:  # a page at a time
                    p = lens[b] - n + done
                    m = min(page - p % page, n - done)
                    y[table[b][p // page], :, p % page:p % page + m] = codes[off[b] + done:off[b] + done + m].transpose(0, 1)
                    done += m
            out += [None, y]
        return out

    def dense(pages, scale, b):
        """Request b's tokens [Hkv, lens[b], D] in 64 bits."""
        ids = torch.tensor(table[b][:-(-lens[b] // page)], device="cuda")
        if scale is None:
            x = pages[ids].double()
        else:
            x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            x = x * torch.exp2(scale[ids].double() - 127).unsqueeze(-1)
        return x.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :lens[b]]

    kv = lambda b: (dense(s["kp"], s["kscale"], b), dense(s["vp"], s["vscale"], b))  # noqa: E731
    if op == "read":
        both = [kv(b) for b in range(B)]
        return [torch.cat([x[i][:, lens[b] - (off[b + 1] - off[b]):].transpose(0, 1) for b, x in enumerate(both)])
                for i in range(2)]
    G = case["G"]
    o = torch.empty(s["rows"], Hkv * G, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["rows"], Hkv * G, dtype=torch.float64, device="cuda")
    for b in range(B):
        k, v = kv(b)
        rows, n = slice(off[b], off[b + 1]), off[b + 1] - off[b]
        ahead = torch.ones(n, lens[b], dtype=torch.bool, device="cuda").triu(lens[b] - n + 1)
        for h in range(Hkv * G):
            x = s["q"][rows, h].double() @ k[h // G].T / math.sqrt(D)
            x = x.masked_fill(ahead, -math.inf)
            lse[rows, h] = torch.logsumexp(x, 1)
            o[rows, h] = torch.softmax(x, 1) @ v[h // G]
    return o, lse
