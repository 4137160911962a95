"""Argument checks of the paged-cache calls (no GPU needed): the C entries return the documented
status before touching CUDA, and the tensor helpers refuse what the library cannot see."""
import pytest
import torch

from attention_forward_sm_gb300 import binding as attn

A = 0x10000  # never dereferenced: every call below fails validation first
NULL, ALIGN, SHAPE = -1, -2, -3
INF, NAN = float("inf"), float("nan")
REQUESTS = dict(table=A, lens=A, offsets=A)
SIZES = dict(B=2, T=8, Hkv=2, D=64, page=16, P=4, M=4)
WRITE = dict(k=A, v=A, k_stride=128, v_stride=128, kpages=A, vpages=A, kscale=0, vscale=0, **REQUESTS, **SIZES)
READ = dict(kpages=A, vpages=A, kscale=0, vscale=0, **REQUESTS, k=A, v=A, **SIZES)
FWD = dict(q=A, q_stride=256, kpages=A, vpages=A, kscale=0, vscale=0, **REQUESTS, o=A, lse=A, B=2, T=8, max_new=4,
           Hq=4, Hkv=2, D=64, page=16, P=4, M=4, causal=1, scale=0.1)
DECODE = dict(q=A, q_stride=256, kpages=A, vpages=A, kscale=0, vscale=0, table=A, lens=A, o=A, lse=A, B=2, Hq=4, Hkv=2,
              D=64, page=16, P=4, M=4, scale=0.1)

CACHE = [(dict(kpages=0), NULL), (dict(vpages=0), NULL), (dict(table=0), NULL), (dict(lens=0), NULL),
         (dict(kscale=A), NULL), (dict(vscale=A), NULL),   # one without the other
         (dict(B=0), SHAPE), (dict(B=65537), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=96), SHAPE), (dict(D=256), SHAPE),
         (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=256), SHAPE), (dict(P=0), SHAPE), (dict(M=0), SHAPE),
         (dict(P=2**30), SHAPE),                           # P * Hkv
         (dict(M=2**17 + 1), SHAPE),                       # M * page
         (dict(kpages=A + 8), ALIGN), (dict(vpages=A + 2), ALIGN), (dict(kscale=A + 8, vscale=A), ALIGN),
         (dict(table=A + 2), ALIGN), (dict(lens=A + 1), ALIGN)]
ROWS = [(dict(T=-1), SHAPE), (dict(T=2**24 + 1), SHAPE), (dict(offsets=A + 2), ALIGN), (dict(k=0), NULL),
        (dict(v=0), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(Hkv=65536), SHAPE)]
ATTEND = [(dict(q=0), NULL), (dict(o=0), NULL), (dict(lse=0), NULL), (dict(q=A + 8), ALIGN), (dict(o=A + 8), ALIGN),
          (dict(lse=A + 4), ALIGN), (dict(scale=-0.5), SHAPE), (dict(scale=INF), SHAPE), (dict(scale=NAN), SHAPE),
          (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=258), SHAPE), (dict(q_stride=255), SHAPE),
          (dict(q_stride=260), SHAPE), (dict(q_stride=2**41), SHAPE)]
CASES = {
    "attn_cache_write": (WRITE, CACHE + ROWS + [(dict(k_stride=127), SHAPE), (dict(v_stride=132), SHAPE),
                                                (dict(k_stride=-128), SHAPE), (dict(v_stride=2**41), SHAPE)]),
    "attn_cache_read": (READ, CACHE + ROWS),
    "attn_paged_fwd": (FWD, CACHE + ATTEND + [
        (dict(offsets=0), NULL), (dict(T=-1), SHAPE), (dict(T=2**24 + 1), SHAPE), (dict(max_new=-1), SHAPE),
        (dict(offsets=A + 2), ALIGN), (dict(T=2**20, Hq=256, M=2**16, q_stride=2**20), SHAPE)]),  # units of work
    "attn_paged_decode": (DECODE, CACHE + ATTEND),
}
ALL = [(fn, change, status) for fn, (_, changes) in CASES.items() for change, status in changes]


@pytest.fixture(scope="module")
def lib():
    from attention_forward_sm_gb300 import _build
    _build.build()
    return attn.load()


@pytest.mark.parametrize("fn,change,status", ALL, ids=[f"{f[5:]}-{','.join(f'{k}={v}' for k, v in c.items())}"
                                                       for f, c, _ in ALL])
def test_refusals(lib, fn, change, status):
    assert getattr(lib, fn)(*{**CASES[fn][0], **change}.values(), None) == status


@pytest.mark.parametrize("fn,change", [("attn_cache_write", dict(T=0, k=0, v=0)), ("attn_cache_read", dict(T=0, k=0, v=0)),
                                       ("attn_paged_fwd", dict(T=0, q=0, o=0, lse=0)),
                                       ("attn_paged_fwd", dict(max_new=0))])
def test_no_rows_are_nothing_to_do(lib, fn, change):
    assert getattr(lib, fn)(*{**CASES[fn][0], **change}.values(), None) == 0


WIDE = [(fn, name) for fn, (case, _) in CASES.items() for name in case
        if name in ("B", "T", "max_new", "Hq", "Hkv", "D", "page", "P", "M")]


@pytest.mark.parametrize("fn,name", WIDE, ids=lambda x: x)
@pytest.mark.parametrize("turns", [1, -1])
def test_sizes_that_only_fit_after_wrapping_are_refused(lib, fn, name, turns):
    """2^32 more or less is the same int in C."""
    case = CASES[fn][0]
    with pytest.raises(attn.AttnError) as e:
        getattr(attn, fn)(**{**case, name: case[name] + turns * 2**32}, stream=0)
    assert e.value.status == SHAPE


@pytest.mark.parametrize("fn,name", [(fn, name) for fn, (case, _) in CASES.items() for name in case if "stride" in name])
def test_strides_beyond_64_bits_are_refused(lib, fn, name):
    with pytest.raises(attn.AttnError) as e:
        getattr(attn, fn)(**{**CASES[fn][0], name: 2**64 + CASES[fn][0][name]}, stream=0)
    assert e.value.status == SHAPE


def _cpu(**change):
    bf16, i32 = torch.bfloat16, torch.int32
    t = dict(kpages=torch.zeros(4, 2, 16, 64, dtype=bf16), vpages=torch.zeros(4, 2, 16, 64, dtype=bf16),
             table=torch.zeros(2, 4, dtype=i32), lens=torch.zeros(2, dtype=i32), offsets=torch.zeros(3, dtype=i32))
    return {**t, **change}


def test_helpers_refuse_what_the_library_cannot_see():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    calls = [lambda **c: attn.cache_write(k, k, **_cpu(**c)), lambda **c: attn.cache_read(**_cpu(**c), rows=2),
             lambda **c: attn.paged_forward(q, **_cpu(**c)),
             lambda **c: attn.paged_decode(q, **{n: x for n, x in _cpu(**c).items() if n != "offsets"})]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
        with pytest.raises(TypeError, match="bfloat16 or float8"):
            call(kpages=torch.zeros(4, 2, 16, 64))
        with pytest.raises(ValueError, match="dimensions"):
            call(table=torch.zeros(2, dtype=torch.int32))
        with pytest.raises(TypeError, match="torch tensor"):
            call(table=[[0]])
    with pytest.raises(TypeError, match="offsets"):
        attn.paged_forward(q, **_cpu(offsets=None))
