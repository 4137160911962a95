"""Cases of the score-modified attention operators and their plain forms.

Four operators of ``attention_forward_sm_gb300``:

* ``fwd``    ``forward_mod``: prefill whose scores are capped by a tanh, biased by
  distance, and masked by a key range per query row (documents, prefixes, padding);
* ``ranges`` ``row_ranges``: those key ranges from document and prefix lengths;
* ``varlen`` ``decode_varlen``: one query token per request, a length per request;
* ``prefix`` ``decode_prefix``: the same for requests that share a long prefix.

Definition, for query row i at position p_i and key j:
x = scale * q_i.k_j;  x = c tanh(x / c) if c > 0;  x = x - m_h |p_i - j| if there are slopes;
O = sum_j softmax(x)_j v_j and LSE = ln sum_j exp(x_j) over the visible keys (none: 0 and -inf).

Lengths are quantiles of a distribution in an order drawn from the seed, so every seed
gives other inputs of the same work.
"""
import math
import statistics

import torch

own = False


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # the smallest call: one short causal prompt, where launch latency is all
        dict(name="fwd tiny", op="fwd", B=1, Hq=2, Hkv=2, N=256, D=64, causal=True, cap=30.0, bias=False,
             docs=0, pad=0, pre=0.0),
        # a long prompt of a model with capped scores, grouped heads
        dict(name="fwd cap 8k", op="fwd", B=1, Hq=32, Hkv=8, N=8192, D=128, causal=True, cap=50.0, bias=False,
             docs=0, pad=0, pre=0.0),
        # prompts packed into rows of 4096 tokens, a tail of padding
        dict(name="fwd documents", op="fwd", B=4, Hq=16, Hkv=16, N=4096, D=128, causal=True, cap=0.0, bias=False,
             docs=7, pad=133, pre=0.0),
        # distance bias, an odd length, the small head
        dict(name="fwd bias odd", op="fwd", B=2, Hq=16, Hkv=16, N=4001, D=64, causal=True, cap=0.0, bias=True,
             docs=0, pad=0, pre=0.0),
        # everything at once: packed documents with a bidirectional prefix each, cap and bias
        dict(name="fwd prefix docs all", op="fwd", B=2, Hq=32, Hkv=8, N=2500, D=128, causal=True, cap=30.0,
             bias=True, docs=3, pad=60, pre=0.25),
        # the mask of one packed batch, and of a very long one with many documents
        dict(name="ranges 4k", op="ranges", B=4, N=4096, causal=True, docs=7, pad=133, pre=0.0),
        dict(name="ranges 128k", op="ranges", B=8, N=131072, causal=True, docs=513, pad=1000, pre=0.25),
        # one request, a short cache: the latency of a decode step
        dict(name="decode one", op="varlen", B=1, Hq=32, Hkv=8, Ncap=2048, lo=1023, hi=1023, D=128, cap=50.0,
             bias=False),
        # a batch whose requests are of very different lengths
        dict(name="decode ragged 64k", op="varlen", B=8, Hq=32, Hkv=8, Ncap=65536, lo=500, hi=65536, D=128,
             cap=50.0, bias=False),
        # few requests on a short shared prompt, all heads on one KV head, odd sizes
        dict(name="prefix few", op="prefix", B=5, Hq=8, Hkv=1, Np=1001, Ncap=256, lo=1, hi=200, D=64, cap=0.0,
             bias=True),
        # a serving batch behind one long system prompt
        dict(name="prefix serving", op="prefix", B=64, Hq=32, Hkv=8, Np=16384, Ncap=1024, lo=16, hi=1024, D=128,
             cap=0.0, bias=False),
        # many samples of one prompt: the shared part is bound by the tensor cores
        dict(name="prefix wide", op="prefix", B=256, Hq=32, Hkv=8, Np=8192, Ncap=512, lo=8, hi=512, D=128,
             cap=50.0, bias=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "ranges", "varlen", "varlen", "prefix", "prefix"])
    if op == "ranges":
        N = _log_int(rng, 64, 131072)
        pad = rng.choice([0, rng.randint(0, N // 8)])
        return dict(op=op, B=rng.randint(1, 8), N=N, causal=rng.random() < 0.8, pad=pad,
                    docs=_log_int(rng, 1, max(1, min(513, (N - pad) // 32))), pre=rng.choice([0.0, 0.25, 0.6]))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 4, 7, 8])
    D = rng.choice([64, 128, 128])
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    bias = rng.random() < 0.4
    if op == "fwd":
        # no more scores than the largest listed case
        N = _log_int(rng, 100, min(8192, int(8192 * math.sqrt(32 / (Hkv * G)))))
        most = max(1, 32 * 8192 * 8192 // (Hkv * G * N * N))
        docs = rng.choice([0, 0, _log_int(rng, 1, max(1, N // 64))])
        return dict(op=op, B=_log_int(rng, 1, min(4, most)), Hq=Hkv * G, Hkv=Hkv, N=N, D=D,
                    causal=rng.random() < 0.8, cap=cap, bias=bias, docs=docs,
                    pad=rng.randint(0, N // 8) if docs else 0, pre=rng.choice([0.0, 0.3]) if docs else 0.0)
    if op == "varlen":
        Ncap = _log_int(rng, 128, 65536)
        B = _log_int(rng, 1, max(1, min(128, 4 * 65536 // Ncap)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Ncap=Ncap, lo=rng.randint(1, max(1, Ncap // 16)), hi=Ncap,
                    D=D, cap=cap, bias=bias)
    B = _log_int(rng, 2, 256)
    Ncap = _log_int(rng, 32, max(32, min(1024, 131072 // B)))
    return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, Np=_log_int(rng, 100, max(100, min(16384, 2097152 // B))),
                Ncap=Ncap, lo=1, hi=Ncap, D=D, cap=cap, bias=bias)


# ----------------------------------------------------------------------------- lengths


def _doc_lens(case):
    """Lengths of the documents of one packed row: log-normal quantiles that fill N - pad tokens."""
    n, total = case["docs"], case["N"] - case["pad"]
    z = [math.exp(0.8 * statistics.NormalDist().inv_cdf((m + 0.5) / n)) for m in range(n)]
    lens = [max(1, int(x / sum(z) * total)) for x in z]
    lens[-1] += total - sum(lens)
    return lens


def _seq_lens(case):
    """One length per request: quantiles of a log-uniform distribution on [lo, hi]."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    return [max(lo, min(hi, round(lo * (hi / lo) ** (b / (B - 1))))) for b in range(B)]


def _visible_pairs(case):
    """Visible (row, key) pairs of one batch row and head of a fwd case."""
    def one(n):
        if not case["causal"]:
            return n * n
        p = int(n * case["pre"])
        return n * (n + 1) // 2 + p * (p - 1) // 2  # rows below the prefix see all of it
    return sum(one(n) for n in (_doc_lens(case) if case["docs"] else [case["N"]]))


def work(case):
    op = case["op"]
    if op == "ranges":
        return {"bytes": case["B"] * (8 * case["N"] + (8 if case["pre"] else 4) * case["docs"]),
                "flops": 4 * case["B"] * case["N"]}
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if op == "fwd":
        N = case["N"]
        return {"bytes": 4 * B * (Hq + Hkv) * N * D + 4 * B * Hq * N + (8 * B * N if case["docs"] else 0),
                "flops": 4 * D * B * Hq * _visible_pairs(case)}
    keys = sum(_seq_lens(case))
    pre = case["Np"] if op == "prefix" else 0
    return {"bytes": 4 * Hkv * D * (keys + pre) + 4 * B * Hq * D + 4 * B * Hq + 4 * B,
            "flops": 4 * D * Hq * (keys + B * pre)}


# ----------------------------------------------------------------------------- inputs


def _normal(gen, shape, sigma=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32, device="cuda") * sigma).to(torch.bfloat16)


def _slopes(case):
    if not case["bias"]:
        return None
    H = case["Hq"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _docs_of(case, gen):
    """[B, docs] document lengths in an order of the seed, and the prefix length of each."""
    order = torch.stack([torch.randperm(case["docs"], generator=gen, device="cuda") for _ in range(case["B"])])
    lens = torch.tensor(_doc_lens(case), dtype=torch.int32, device="cuda")[order]
    return lens, (lens.double() * case["pre"]).to(torch.int32) if case["pre"] else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * int(seed) + 17)
    s = dict(case)
    op = case["op"]
    if op == "ranges":
        s["lens"], s["prefix"] = _docs_of(case, gen)
        return s
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    # capped models have wide scores (standard deviation 6 here, so that the cap bites), others about 1
    sigma = 6.0 if case["cap"] else 1.0
    s["slopes"] = _slopes(case)
    if op == "fwd":
        N = case["N"]
        s["q"] = _normal(gen, (B, Hq, N, D), sigma)
        s["k"] = _normal(gen, (B, Hkv, N, D))
        s["v"] = _normal(gen, (B, Hkv, N, D))
        s["ranges"] = None
        if case["docs"]:  # the mask of the batch, made once and used by every layer
            lens, pre = _docs_of(case, gen)
            s["ranges"] = _plain_ranges(lens, pre, N, case["causal"])
        return s
    s["q"] = _normal(gen, (B, Hq, D), sigma)
    s["k"] = _normal(gen, (B, Hkv, case["Ncap"], D))
    s["v"] = _normal(gen, (B, Hkv, case["Ncap"], D))
    order = torch.randperm(B, generator=gen, device="cuda")
    s["lens"] = torch.tensor(_seq_lens(case), dtype=torch.int32, device="cuda")[order]
    if op == "prefix":
        s["pk"] = _normal(gen, (Hkv, case["Np"], D))
        s["pv"] = _normal(gen, (Hkv, case["Np"], D))
    return s


# ----------------------------------------------------------------------------- plain forms


def _plain_ranges(lens, pre, N, causal):
    ends = lens.long().cumsum(1)  # [B, M]
    i = torch.arange(N, device=lens.device).expand(lens.shape[0], N).contiguous()
    m = torch.searchsorted(ends, i, right=True)  # the first document that ends after i
    inside = m < lens.shape[1]
    m = m.clamp(max=lens.shape[1] - 1)
    hi = ends.gather(1, m)
    lo = hi - lens.long().gather(1, m)
    if causal:
        last = i + 1
        if pre is not None:
            last = torch.maximum(last, torch.minimum(lo + pre.long().gather(1, m), hi))
        hi = last
    return torch.where(inside.unsqueeze(-1), torch.stack([lo, hi], -1), 0).to(torch.int32)


def _scores(x, dist, cap, slopes):
    """Cap and bias: x [B, H, rows, keys], dist broadcastable to it."""
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    if slopes is not None:
        x = x - (slopes.view(1, -1, 1, 1).double() * dist).float()
    return x


def _attend(x, v):
    """softmax(x) v with -inf as masked; rows that see nothing give 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain_fwd(s):
    B, Hq, N, D = s["q"].shape
    G = Hq // s["k"].shape[1]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    x = torch.matmul(q.view(B, -1, G * N, D), k.transpose(2, 3)).view(B, Hq, N, N) / math.sqrt(D)
    i = torch.arange(N, device=q.device)
    x = _scores(x, (i[:, None] - i[None, :]).abs(), s["cap"], s["slopes"])
    if s["ranges"] is not None:
        r = s["ranges"]
        seen = (i >= r[..., 0:1]) & (i < r[..., 1:2])  # [B, N, N]
        x = torch.where(seen.unsqueeze(1), x, -math.inf)
    elif s["causal"]:
        x = torch.where(i[None, :] <= i[:, None], x, -math.inf)
    o, lse = _attend(x.view(B, -1, G * N, N), v)
    return o.view(B, Hq, N, D), lse.view(B, Hq, N)


def _plain_decode(s):
    B, Hq, D = s["q"].shape
    k, v = s["k"].float(), s["v"].float()
    Hkv, n = k.shape[1], k.shape[2]
    G = Hq // Hkv
    q = s["q"].float().view(B, Hkv, G, D)
    j = torch.arange(n, device=q.device)
    lens = s["lens"].long().view(B, 1, 1, 1)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hq, 1, n) / math.sqrt(D)
    x = _scores(x, (lens - 1 - j).abs(), s["cap"], s["slopes"])
    x = torch.where(j < lens, x, -math.inf)
    if s["op"] == "varlen":
        o, lse = _attend(x.view(B, Hkv, G, n), v)
        return o.view(B, Hq, D), lse.view(B, Hq)
    # the shared keys once for the whole batch: rows (b, g) of a KV head in one product
    pk, pv = s["pk"].float(), s["pv"].float()
    Np = pk.shape[1]
    rows = q.transpose(0, 1).reshape(Hkv, B * G, D)
    y = torch.matmul(rows, pk.transpose(1, 2)).view(Hkv, B, G, Np).transpose(0, 1).reshape(B, Hq, 1, Np) / math.sqrt(D)
    y = _scores(y, Np + lens - 1 - torch.arange(Np, device=q.device), s["cap"], s["slopes"])
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    px, py = torch.exp(x - m), torch.exp(y - m)
    total = px.sum(-1) + py.sum(-1)  # [B, Hq, 1]
    o = torch.matmul(px.view(B, Hkv, G, n), v).view(B, Hq, D)
    oy = torch.matmul(py.view(B, Hkv, G, Np).transpose(0, 1).reshape(Hkv, B * G, Np), pv)
    o = o + oy.view(Hkv, B, G, D).transpose(0, 1).reshape(B, Hq, D)
    return (o / total).to(torch.bfloat16), (m.squeeze(-1) + torch.log(total)).view(B, Hq)


def run(state):
    s = state
    if own:
        import attention_forward_sm_gb300 as attn
        if s["op"] == "ranges":
            return attn.row_ranges(s["lens"], s["N"], prefix_lens=s["prefix"], causal=s["causal"])
        if s["op"] == "fwd":
            # the ranges of a causal batch hold the causal limit already
            return attn.forward_mod(s["q"], s["k"], s["v"], causal=s["causal"] and s["ranges"] is None,
                                    softcap=s["cap"], slopes=s["slopes"], ranges=s["ranges"])
        if s["op"] == "varlen":
            return attn.decode_varlen(s["q"], s["k"], s["v"], s["lens"], softcap=s["cap"], slopes=s["slopes"])
        return attn.decode_prefix(s["q"], s["pk"], s["pv"], s["k"], s["v"], s["lens"], softcap=s["cap"],
                                  slopes=s["slopes"])
    if s["op"] == "ranges":
        return _plain_ranges(s["lens"], s["prefix"], s["N"], s["causal"])
    return _plain_fwd(s) if s["op"] == "fwd" else _plain_decode(s)


# ----------------------------------------------------------------------------- 64 bits


def _exact_rows(q, k, v, pos, jpos, seen, cap, slope):
    """Attention of rows q [R, D] over keys k [n, D] in 64 bits."""
    x = (q.double() @ k.double().T) * (1.0 / math.sqrt(q.shape[1]))
    if cap > 0:
        e = torch.exp(-2.0 * x.abs() / cap)
        x = torch.sign(x) * cap * (1 - e) / (1 + e)
    if slope is not None:
        x = x - slope.double() * (pos.double()[:, None] - jpos.double()[None, :]).abs()
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return w @ v.double(), lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ranges":
        return None  # whole numbers
    B, Hq, D = case["B"], case["Hq"], case["D"]
    G = Hq // case["Hkv"]
    slope = lambda h: None if s["slopes"] is None else s["slopes"][h]  # noqa: E731
    if case["op"] == "fwd":
        N = case["N"]
        o = torch.empty(B, Hq, N, D, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, Hq, N, dtype=torch.float64, device="cuda")
        j = torch.arange(N, device="cuda")
        for b in range(B):
            if s["ranges"] is not None:
                seen = (j[None, :] >= s["ranges"][b, :, :1]) & (j[None, :] < s["ranges"][b, :, 1:])
            else:
                seen = j[None, :] <= (j[:, None] if case["causal"] else j[-1])
                seen = seen.expand(N, N)
            for h in range(Hq):
                o[b, h], lse[b, h] = _exact_rows(s["q"][b, h], s["k"][b, h // G], s["v"][b, h // G], j, j, seen,
                                                 case["cap"], slope(h))
        return o, lse
    o = torch.empty(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Hq, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(B):
        for kv in range(case["Hkv"]):
            k, v = s["k"][b, kv, :lens[b]], s["v"][b, kv, :lens[b]]
            if case["op"] == "prefix":
                k, v = torch.cat([s["pk"][kv], k]), torch.cat([s["pv"][kv], v])
            j = torch.arange(k.shape[0], device="cuda")
            heads = slice(kv * G, (kv + 1) * G)
            seen = torch.ones(G, k.shape[0], dtype=torch.bool, device="cuda")
            slopes = None if s["slopes"] is None else s["slopes"][heads, None]
            o[b, heads], lse[b, heads] = _exact_rows(s["q"][b, heads], k, v, j[-1:].expand(G), j, seen, case["cap"],
                                                     slopes)
    return o, lse
