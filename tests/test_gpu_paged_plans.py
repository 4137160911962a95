"""Paged attention where its plans have to do more than in an ordinary batch: several blocks of
rows of a request in the kernel for few rows (a table wider than 2^18 tokens), more requests than
a block has threads, requests without new tokens among them."""
import pytest

torch = pytest.importorskip("torch")

import paged_ref as ref  # noqa: E402
from attention_forward_sm_gb300 import binding as attn  # noqa: E402
from test_gpu_paged import _randn  # noqa: E402
from test_gpu_paged_range import check_range  # noqa: E402

pytestmark = pytest.mark.gpu
QUANT = pytest.mark.parametrize("quant", [False, True], ids=["bf16", "e4m3"])


def _widen(c, tokens):
    """The cache with a table of so many tokens a request, out of range behind its pages."""
    table = torch.full((len(c.lens), tokens // c.page), -7, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    c.table = table


@QUANT
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,new,G", [([300, 77, 0, 1000], [70, 77, 0, 9], 4), ([2000], [500], 1), ([40, 700], [3, 50], 7),
                                        ([130], [2], 128)])
def test_wide_tables(quant, D, page, causal, lens, new, G):
    c = ref.Cache(lens, 2, D, page, quant, seed=21)
    _widen(c, 2 ** 19)
    offsets = ref.offsets_of(new)
    q = _randn((sum(new), 2 * G, D), 22)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=max(new), causal=causal, **c.scales())
    check_range(o, lse, q, c, offsets, causal=causal)
    # a bound on the new tokens that is too small decides nothing but the layout
    again = attn.paged_forward(q, *c.args(), offsets, max_new=1, causal=causal, **c.scales())
    check_range(*again, q, c, offsets, causal=causal)


@QUANT
@pytest.mark.parametrize("page", [64, 128])
def test_more_than_a_segment_of_keys(quant, page):
    """A cache of more than 2^18 tokens, chunks of several blocks of rows."""
    c = ref.Cache([2 ** 18 + 333, 50], 1, 64, page, quant, seed=23)
    offsets = ref.offsets_of([41, 30])
    q = _randn((71, 2, 64), 24)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=41, **c.scales())
    check_range(o, lse, q, c, offsets)


@QUANT
@pytest.mark.parametrize("B", [700, 1700])
@pytest.mark.parametrize("most", [3, 40])
def test_more_requests_than_threads(quant, B, most):
    g = torch.Generator().manual_seed(B + most)
    lens = torch.randint(0, 50, (B,), generator=g)
    new = torch.randint(0, 4, (B,), generator=g)
    new[torch.rand(B, generator=g) < 0.5] = 0
    new[-3:] = 0
    new[B // 3], lens[B // 3] = most, 600
    new = torch.minimum(new, lens).tolist()
    # (requests that share the pages of a few)
    c = ref.Cache([50] * 20 + [600], 1, 64, 16, quant, seed=25)
    of = [20 if n == 600 else b % 20 for b, n in enumerate(lens.tolist())]
    c.table, c.lens_t, c.lens = c.table[of].contiguous(), lens.int().cuda(), lens.tolist()
    c.dense = [tuple(x[:n] for x in c.dense[i]) for i, n in zip(of, c.lens)]
    offsets = ref.offsets_of(new)
    q = _randn((sum(new), 4, 64), 26)
    o, lse = attn.paged_forward(q, *c.args(), offsets, max_new=most, **c.scales())
    check_range(o, lse, q, c, offsets)
    if most == 3:
        q = _randn((B, 4, 64), 27)
        o, lse = attn.paged_decode(q, *c.args(), **c.scales())
        some = [b for b in range(B) if lens[b] > 0]
        none = [b for b in range(B) if lens[b] == 0]
        assert not o[none].any() and torch.isinf(lse[none]).all()
        c.lens, c.dense, c.table = [c.lens[b] for b in some], [c.dense[b] for b in some], c.table[some]
        check_range(o[some], lse[some], q[some], c, ref.offsets_of([1] * len(some)))
