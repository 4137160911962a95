"""Paged caches as a server uses them: written, attended and read back step by step, captured
in graphs, on several streams, in pools beyond 32-bit offsets; and refusals on the GPU."""
import math
import threading

import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402
from attention_forward_sm_gb300 import binding as attn  # noqa: E402
from test_gpu_paged import _randn, check_attention  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, E4M3 = ref.BF16, ref.E4M3


def _pool(P, Hkv, page, D, quant):
    kp, vp = (torch.zeros(P, Hkv, page, D, dtype=BF16, device="cuda").to(E4M3 if quant else BF16) for _ in range(2))
    if not quant:
        return dict(kpages=kp, vpages=vp)
    ks, vs = (torch.full((P, Hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    return dict(kpages=kp, vpages=vp, kscale=ks, vscale=vs)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
def test_prompts_in_chunks_then_tokens(quant):
    """Three requests, one of which comes later: chunks of their prompts and single tokens in
    the same batches, each step writing, then attending.  Every row against dense attention over
    what the cache then gives back, the whole cache against what went in."""
    Hkv, G, D, page, M = 2, 3, 64, 16, 16
    Hq = Hkv * G
    total = [70, 200, 33]
    plan = [[40, 100, 0], [30, 90, 0], [0, 1, 30], [0, 1, 1], [0, 8, 1], [0, 0, 1]]
    assert [sum(s[b] for s in plan) for b in range(3)] == total
    pool = _pool(3 * M, Hkv, page, D, quant)
    table = _i32([[M * b + (7 * i + b) % M for i in range(M)] for b in range(3)])
    x = [_randn((n, Hq + 2 * Hkv, D), 40 + b) for b, n in enumerate(total)]
    done = [0, 0, 0]
    rows = [([], []) for _ in total]
    scales = {k: v for k, v in pool.items() if "scale" in k}
    for step in plan:
        new = torch.cat([x[b][done[b]:done[b] + n] for b, n in enumerate(step)])
        done = [d + n for d, n in zip(done, step)]
        lens, offsets = _i32(done), ref.offsets_of(step)
        q, k, v = new[:, :Hq], new[:, Hq:Hq + Hkv], new[:, Hq + Hkv:]
        attn.cache_write(k, v, pool["kpages"], pool["vpages"], table, lens, offsets, **scales)
        o, lse = attn.paged_forward(q, pool["kpages"], pool["vpages"], table, lens, offsets, max_new=max(step), **scales)
        at = 0
        for b, n in enumerate(step):
            rows[b][0].append(o[at:at + n])
            rows[b][1].append(lse[at:at + n])
            at += n
    k, v = attn.cache_read(pool["kpages"], pool["vpages"], table, _i32(total), ref.offsets_of(total), sum(total), **scales)
    at = 0
    for b, n in enumerate(total):
        kb, vb = k[at:at + n], v[at:at + n]
        at += n
        for got, put in ((kb, x[b][:, Hq:Hq + Hkv]), (vb, x[b][:, Hq + Hkv:])):
            if quant:  # half a step of e4m3 relative to the value, or of its smallest numbers
                scale = put.float().abs().amax(-1, keepdim=True) / 224
                assert ((got.float() - put.float()).abs() <= 2.0 ** -4 * put.float().abs() + 2.0 ** -10 * scale).all()
            else:
                assert torch.equal(got, put)
        c = ref.Cache([0], Hkv, D, page, False)
        c.lens, c.dense = [n], [(kb.double(), vb.double())]
        check_attention(torch.cat(rows[b][0]), torch.cat(rows[b][1]), x[b][:, :Hq], c, ref.offsets_of([n]))
        # (the dense prefill of this framework gives the same, up to both roundings)
        o, lse = attn.forward(*(y.transpose(0, 1).contiguous()[None] for y in (x[b][:, :Hq], kb, vb)), causal=True)
        far = (o[0].transpose(0, 1).float() - torch.cat(rows[b][0]).float()).abs().max()
        assert float(far) <= 2 * 2.0 ** -7 * float(vb.float().abs().max())
    assert attn.attn_get_device_error() == 0


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_captured_and_replayed(quant, new):
    """Two graphs of a step each, replayed in turn with other lengths, between eager calls."""
    Hkv, G, D, page, B, M = 2, 4, 128, 32, 3, 40
    pool = _pool(B * M, Hkv, page, D, quant)
    scales = {k: v for k, v in pool.items() if "scale" in k}
    table = _i32([[B * i + b for i in range(M)] for b in range(B)])
    c = ref.Cache([M * page] * B, Hkv, D, page, quant, seed=20, spare=0)
    for b in range(B):  # the reference's pages, at this test's places
        for i in range(M):
            for name, src in (("kpages", c.kp), ("vpages", c.vp), ("kscale", c.ks), ("vscale", c.vs)):
                if src is not None:
                    d, s = pool[name], src
                    if d.dtype == E4M3:
                        d, s = d.view(torch.uint8), s.view(torch.uint8)
                    d[B * i + b] = s[int(c.table[b, i])]
    lens, offsets = _i32([new] * B), ref.offsets_of([new] * B)
    q = _randn((B * new, Hkv * G, D), 21)

    def step():
        return attn.paged_forward(q, pool["kpages"], pool["vpages"], table, lens, offsets, max_new=new, **scales)

    def check(out, n):
        d = ref.Cache([0], Hkv, D, page, False)
        d.lens, d.dense = list(n), [(k[:m], v[:m]) for (k, v), m in zip(c.dense, n)]
        check_attention(*out, q, d, offsets)

    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for i, n in enumerate([[1280, 900, new], [new, new, new], [700, 1280, 33 + new], [1280, 1280, 1280], [64, 128, 65 + new]]):
        lens.copy_(_i32(n))
        g, out = graphs[i % 2]
        g.replay()
        eager = step()
        g.replay()
        check(out, n)
        check(eager, n)
        graphs[(i + 1) % 2][0].replay()
        check(graphs[(i + 1) % 2][1], n)
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])


def test_calls_in_any_order_on_any_stream():
    """Calls of different sizes and types (other kernels, other numbers of CTAs) share their
    stream's buffer; ten streams and threads at once, more than there are buffers."""
    cases = []
    for i, (quant, G, new, lens) in enumerate([(False, 4, 1, [3000, 70]), (True, 8, 1, [5000, 20, 900]), (True, 4, 4, [4000]),
                                               (False, 4, 30, [2000, 600]), (True, 2, 90, [2500]), (False, 16, 1, [777, 8000])]):
        c = ref.Cache(lens, 4, 128, 64, quant, seed=30 + i)
        offsets = ref.offsets_of([new] * len(lens))
        q = _randn((new * len(lens), 4 * G, 128), 31 + i)
        want = attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
        check_attention(*want, q, c, offsets)
        cases.append((q, c, offsets, new, want))
    torch.cuda.synchronize()
    wrong = []

    def work(seed, stream):
        order = torch.randperm(60, generator=torch.Generator().manual_seed(seed)) % len(cases)
        for i in order.tolist():
            q, c, offsets, new, want = cases[i]
            got = attn.paged_forward(q, *c.args(), offsets, max_new=new, stream=stream, **c.scales())
            stream.synchronize()
            if not (torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])):
                wrong.append((seed, i))

    streams = [torch.cuda.Stream() for _ in range(10)]
    threads = [threading.Thread(target=work, args=(i, s)) for i, s in enumerate(streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    # and one after another on one stream, nothing waited for in between
    got = [attn.paged_forward(q, *c.args(), offsets, max_new=new, **c.scales())
           for _ in range(3) for q, c, offsets, new, _ in cases]
    for i, g in enumerate(got):
        assert torch.equal(g[0], cases[i % len(cases)][4][0])
    assert attn.attn_get_device_error() == 0


def test_other_streams():
    """Writes, reads and attention queued on another stream than the current one."""
    c = ref.Cache([200, 90], 2, 64, 32, True, seed=50)
    offsets = ref.offsets_of([3, 5])
    kv = _randn((8, 4, 64), 51)
    q = _randn((8, 4, 64), 52)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    attn.cache_write(kv[:, :2], kv[:, 2:], c.kp, c.vp, c.table, c.lens_t, offsets, stream=s, **c.scales())
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=5, stream=s, **c.scales())
    k, v = attn.cache_read(c.kp, c.vp, c.table, c.lens_t, ref.offsets_of(c.lens), 290, stream=s, **c.scales())
    torch.cuda.current_stream().wait_stream(s)
    c.dense = [(k[:200].double(), v[:200].double()), (k[200:].double(), v[200:].double())]
    check_attention(o, lse, q, c, offsets)
    codes, e = ref.quantise(kv[:3, :2])
    assert torch.equal(k[197:200].double(), codes * torch.exp2(e.double()).unsqueeze(-1))


@pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 60])
def test_pools_beyond_32_bit_offsets(quant, new):
    """Pages on either side of 2^31 and 2^32 elements (and bytes) of a pool."""
    Hkv, D, page = 8, 128, 128
    each = Hkv * page * D  # elements of a page
    P = (2**32 + 2**28) // each
    pool = dict(kpages=torch.empty(P, Hkv, page, D, dtype=E4M3 if quant else BF16, device="cuda"),
                vpages=torch.empty(P, Hkv, page, D, dtype=E4M3 if quant else BF16, device="cuda"))
    scales = {}
    if quant:
        scales = {n: torch.empty(P, Hkv, page, dtype=torch.uint8, device="cuda") for n in ("kscale", "vscale")}
    ids = [0, 2**31 // each - 1, 2**31 // each, P - 1, 2**30 // each, 2**32 // each]
    n = len(ids) * page - 50
    table, lens = _i32([ids]), _i32([n])
    kv = _randn((n, 2 * Hkv, D), 60)
    attn.cache_write(kv[:, :Hkv], kv[:, Hkv:], **pool, table=table, lens=lens, offsets=_i32([0, n]), **scales)
    k, v = attn.cache_read(**pool, table=table, lens=lens, offsets=_i32([0, n]), rows=n, **scales)
    if not quant:
        assert torch.equal(k, kv[:, :Hkv]) and torch.equal(v, kv[:, Hkv:])
    c = ref.Cache([0], Hkv, D, page, False)
    c.lens, c.dense = [n], [(k.double(), v.double())]
    q = _randn((new, 2 * Hkv, D), 61)
    o, lse = attn.paged_forward(q, **pool, table=table, lens=lens, offsets=_i32([0, new]), max_new=new, **scales)
    check_attention(o, lse, q, c, ref.offsets_of([new]))


def test_lengths_and_offsets_are_clamped():
    """Whatever stands in lens and offsets, nothing out of bounds is read or written."""
    for quant in (False, True):
        c = ref.Cache([64, 48], 2, 64, 16, quant, seed=70)
        good = [c.kp.clone(), c.vp.clone()]
        q = _randn((20, 4, 64), 71)
        kv = _randn((20, 4, 64), 72)
        for lens, offsets in [([2**31 - 1, -5], [0, 10, 20]), ([64, 48], [-7, 2**31 - 1, 5]), ([64, 48], [20, 0, -2**31]),
                              ([-2**31, 64], [5, 5, 5]), ([1, 1], [0, 2**31 - 1, 2**31 - 1])]:
            lens, offsets = _i32(lens), _i32(offsets)
            attn.paged_forward(q, c.kp, c.vp, c.table, lens, offsets, max_new=20, **c.scales())
            attn.paged_forward(q, c.kp, c.vp, c.table, lens, offsets, max_new=2, **c.scales())
            attn.cache_read(c.kp, c.vp, c.table, lens, offsets, 20, **c.scales())
            attn.cache_write(kv[:, :2], kv[:, 2:], c.kp, c.vp, c.table, lens, offsets, **c.scales())
            torch.cuda.synchronize()
            assert attn.attn_get_device_error() in (0, 0x40)  # (entries of the table out of range)
        used = set(c.table[0].tolist() + c.table[1, :3].tolist())
        for p in range(c.kp.shape[0]):
            if p not in used:
                assert torch.equal(c.kp[p].view(torch.uint8), good[0][p].view(torch.uint8))
                assert torch.equal(c.vp[p].view(torch.uint8), good[1][p].view(torch.uint8))


def test_empty_calls():
    c = ref.Cache([5, 0], 2, 64, 16, False, seed=80)
    none = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    offsets = _i32([0, 0, 0])
    o, lse = attn.paged_forward(none, *c.args(), offsets)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    attn.cache_write(none[:, :2], none[:, :2], *c.args(), offsets)
    k, v = attn.cache_read(*c.args(), offsets, 0)
    assert k.shape == v.shape == (0, 2, 64)


def test_helpers_refuse_on_the_gpu():
    c = ref.Cache([40, 20], 2, 64, 16, True, seed=90)
    b = ref.Cache([40, 20], 2, 64, 16, False, seed=90)
    q = _randn((2, 4, 64), 91)
    kv = _randn((2, 2, 64), 92)
    with pytest.raises(ValueError, match="need kscale"):
        attn.paged_decode(q, *c.args())
    with pytest.raises(ValueError, match="no kscale"):
        attn.paged_decode(q, *b.args(), **c.scales())
    with pytest.raises(ValueError, match="kscale must have shape"):
        attn.paged_decode(q, *c.args(), kscale=c.ks[1:], vscale=c.vs)
    with pytest.raises(TypeError, match="uint8"):
        attn.paged_decode(q, *c.args(), kscale=c.ks.int(), vscale=c.vs)
    with pytest.raises(TypeError, match="int32"):
        attn.paged_decode(q, b.kp, b.vp, b.table.long(), b.lens_t)
    with pytest.raises(ValueError, match="lens must have shape"):
        attn.paged_decode(q, b.kp, b.vp, b.table, b.lens_t[:1])
    with pytest.raises(ValueError, match="contiguous"):
        attn.paged_decode(q, b.kp.transpose(1, 2), b.vp.transpose(1, 2), b.table, b.lens_t)
    with pytest.raises(ValueError, match="inconsistent B"):
        attn.paged_decode(_randn((3, 4, 64), 1), *b.args())
    with pytest.raises(ValueError, match="must have shape"):
        attn.paged_decode(_randn((2, 4, 128), 1), *b.args())
    with pytest.raises(ValueError, match="heads of a token"):
        attn.paged_decode(_randn((2, 4, 128), 1)[..., ::2], *b.args())
    with pytest.raises(TypeError, match="bfloat16"):
        attn.paged_decode(q.float(), *b.args())
    with pytest.raises(ValueError, match="must have shape"):
        attn.cache_write(_randn((2, 3, 64), 1), kv, *b.args())
    with pytest.raises(ValueError, match="inconsistent T"):
        attn.cache_write(kv, kv[:1], *b.args(), ref.offsets_of([1, 1]))
    with pytest.raises(ValueError, match="rows must be given"):
        attn.cache_read(*b.args(), ref.offsets_of([1, 1]))
    with pytest.raises(attn.AttnError):
        attn.paged_decode(_randn((2, 3, 64), 1), *b.args())       # 3 query heads on 2
    with pytest.raises(attn.AttnError):
        attn.paged_decode(q, *b.args(), scale=math.nan)
    with pytest.raises(attn.AttnError):                            # a stride of no multiple of 8
        attn.paged_decode(_randn((2, 260), 1)[:, :256].view(2, 4, 64), *b.args())
    kp = torch.zeros(4, 2, 24, 64, dtype=BF16, device="cuda")
    with pytest.raises(attn.AttnError):                            # pages of 24 tokens
        attn.paged_decode(q, kp, kp, b.table, b.lens_t)


def test_a_thread_s_first_call():
    """In threads that have made no CUDA call yet, with all outputs out of torch's cache."""
    c = ref.Cache([200, 90], 2, 64, 32, False, seed=95)
    q = _randn((2, 4, 64), 96)
    qn = _randn((100, 4, 64), 97)
    offsets = ref.offsets_of([40, 60])
    calls = [lambda: attn.paged_decode(q, *c.args()), lambda: attn.paged_forward(qn, *c.args(), offsets)]
    wants = [[f() for _ in range(3)][0] for f in calls]
    torch.cuda.synchronize()
    found = []

    def work(i):
        try:
            found.append(all(torch.equal(a, b) for a, b in zip(calls[i % 2](), wants[i % 2])))
        except Exception as e:  # noqa: BLE001
            found.append(e)

    for i in range(12):
        t = threading.Thread(target=work, args=(i,))
        t.start()
        t.join()
    assert found == [True] * 12
