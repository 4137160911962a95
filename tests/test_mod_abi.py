"""Argument checks of the calls with modified scores (no GPU needed): the C
entries return the documented status before touching CUDA, and the tensor
helpers refuse what the library cannot see."""
import pytest
import torch

from attention_forward_sm_gb300 import binding as attn

A = 0x10000  # never dereferenced: every call below fails validation first
OK_FWD = dict(q=A, k=A, v=A, o=A, lse=A, B=1, Hq=4, Hkv=2, Nq=8, Nk=8, D=64, causal=1, q_offset=0,
              scale=0.1, softcap=0.0, slopes=0, ranges=0)
OK_RANGES = dict(doc_lens=A, prefix_lens=0, ranges=A, B=1, N=8, M=2, causal=1)
OK_VARLEN = dict(q=A, kcache=A, vcache=A, lens=A, o=A, lse=A, B=1, Hq=4, Hkv=2, Ncap=16, D=64,
                 scale=0.1, softcap=0.0, slopes=0)
OK_PREFIX = dict(q=A, kprefix=A, vprefix=A, kcache=A, vcache=A, lens=A, o=A, lse=A, B=1, Hq=4, Hkv=2,
                 Np=16, Ncap=16, D=64, scale=0.1, softcap=0.0, slopes=0)
NULL, ALIGN, SHAPE = -1, -2, -3
INF, NAN = float("inf"), float("nan")

SCORE = [(dict(scale=-0.5), SHAPE), (dict(scale=INF), SHAPE), (dict(scale=NAN), SHAPE),
         (dict(softcap=-1.0), SHAPE), (dict(softcap=NAN), SHAPE), (dict(softcap=INF), SHAPE),
         (dict(softcap=1e-45), SHAPE),   # scale / softcap overflows
         (dict(softcap=3e38), SHAPE),    # softcap * log2(e) overflows
         (dict(slopes=A + 2), ALIGN)]
DECODE = [(dict(B=0), SHAPE), (dict(Hq=3), SHAPE), (dict(Hkv=0), SHAPE), (dict(Ncap=0), SHAPE),
          (dict(Ncap=2**30 + 1), SHAPE), (dict(D=96), SHAPE),
          (dict(B=2000, Ncap=2**19), SHAPE),        # more than 12e6 key tiles
          (dict(Hq=258, Hkv=2), SHAPE),             # more than 128 query heads on a KV head
          (dict(Hq=70000, Hkv=70000), SHAPE), (dict(B=2**20, Hkv=2), SHAPE),
          (dict(q=A + 8), ALIGN), (dict(kcache=A + 2), ALIGN), (dict(vcache=A + 4), ALIGN),
          (dict(o=A + 8), ALIGN), (dict(lse=A + 4), ALIGN), (dict(lens=A + 2), ALIGN),
          (dict(q=0), NULL), (dict(kcache=0), NULL), (dict(vcache=0), NULL), (dict(o=0), NULL),
          (dict(lse=0), NULL)]


@pytest.fixture(scope="module")
def lib():
    from attention_forward_sm_gb300 import _build
    _build.build()
    return attn.load()


def _ids(cases):
    return [",".join(f"{k}={v}" for k, v in c[0].items()) for c in cases]


FWD = SCORE + [
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(o=0), NULL), (dict(lse=0), NULL),
    (dict(B=0), SHAPE), (dict(Hq=3), SHAPE), (dict(Hkv=0), SHAPE), (dict(Nq=0), SHAPE),
    (dict(Nk=0), SHAPE), (dict(Nk=2**31 - 1), SHAPE), (dict(D=80), SHAPE), (dict(q_offset=-1), SHAPE),
    (dict(q_offset=2**31 - 1000), SHAPE), (dict(B=2**20, Hq=2**12), SHAPE),
    (dict(q=A + 8), ALIGN), (dict(o=A + 8), ALIGN), (dict(lse=A + 4), ALIGN), (dict(ranges=A + 4), ALIGN)]


@pytest.mark.parametrize("change,status", FWD, ids=_ids(FWD))
def test_fwd_mod_refusals(lib, change, status):
    assert lib.attn_fwd_mod(*{**OK_FWD, **change}.values(), None) == status


RANGES = [(dict(doc_lens=0), NULL), (dict(ranges=0), NULL), (dict(B=0), SHAPE), (dict(B=65536), SHAPE),
          (dict(N=0), SHAPE), (dict(N=2**30 + 1), SHAPE), (dict(M=0), SHAPE),
          (dict(M=2**30 + 1), SHAPE), (dict(B=2048, N=2**30), SHAPE), (dict(ranges=A + 4), ALIGN),
          (dict(doc_lens=A + 1), ALIGN), (dict(prefix_lens=A + 2), ALIGN)]


@pytest.mark.parametrize("change,status", RANGES, ids=_ids(RANGES))
def test_row_ranges_refusals(lib, change, status):
    assert lib.attn_row_ranges(*{**OK_RANGES, **change}.values(), None) == status


@pytest.mark.parametrize("change,status", SCORE + DECODE, ids=_ids(SCORE + DECODE))
def test_decode_varlen_refusals(lib, change, status):
    assert lib.attn_decode_varlen(*{**OK_VARLEN, **change}.values(), None) == status


PREFIX = SCORE + DECODE + [(dict(kprefix=0), NULL), (dict(vprefix=0), NULL), (dict(Np=0), SHAPE),
                           (dict(Np=2**30 + 1), SHAPE), (dict(Np=2**28, B=2000), SHAPE), (dict(kprefix=A + 8), ALIGN),
                           (dict(vprefix=A + 8), ALIGN)]


@pytest.mark.parametrize("change,status", PREFIX, ids=_ids(PREFIX))
def test_decode_prefix_refusals(lib, change, status):
    assert lib.attn_decode_prefix(*{**OK_PREFIX, **change}.values(), None) == status


def test_helpers_refuse_what_the_library_cannot_see():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    q1 = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.forward_mod(x, x, x)
    with pytest.raises(TypeError, match="bfloat16"):
        attn.forward_mod(x.float(), x, x)
    with pytest.raises(ValueError, match="dimensions"):
        attn.forward_mod(x[0], x, x)
    with pytest.raises(ValueError, match="CUDA"):
        attn.decode_varlen(q1, x, x)
    with pytest.raises(ValueError, match="dimensions"):
        attn.decode_prefix(q1, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        attn.row_ranges(torch.zeros(1, 2, dtype=torch.int32), 8)
    with pytest.raises(TypeError, match="int32"):
        attn.row_ranges(torch.zeros(1, 2), 8)
    with pytest.raises(TypeError, match="torch tensor"):
        attn.row_ranges([[1, 2]], 8)


WIDE = [(fn, name) for fn, case in (("attn_fwd_mod", OK_FWD), ("attn_row_ranges", OK_RANGES),
                                    ("attn_decode_varlen", OK_VARLEN), ("attn_decode_prefix", OK_PREFIX))
        for name in case if name in ("B", "Hq", "Hkv", "Nq", "Nk", "Ncap", "Np", "N", "M", "D", "q_offset")]


@pytest.mark.parametrize("fn,name", WIDE, ids=lambda x: x)
@pytest.mark.parametrize("turns", [1, -1])
def test_sizes_that_only_fit_after_wrapping_are_refused(lib, fn, name, turns):
    """2^32 more or less is the same int in C."""
    case = {"attn_fwd_mod": OK_FWD, "attn_row_ranges": OK_RANGES, "attn_decode_varlen": OK_VARLEN,
            "attn_decode_prefix": OK_PREFIX}[fn]
    with pytest.raises(attn.AttnError) as e:
        getattr(attn, fn)(**{**case, name: case[name] + turns * 2**32}, stream=0)
    assert e.value.status == SHAPE


@pytest.mark.parametrize("fn,case", [("attn_fwd_mod", OK_FWD), ("attn_decode_varlen", OK_VARLEN),
                                     ("attn_decode_prefix", OK_PREFIX)], ids=lambda x: x if isinstance(x, str) else "")
def test_caps_that_a_float_rounds_to_none_are_refused(lib, fn, case):
    with pytest.raises(attn.AttnError) as e:
        getattr(attn, fn)(**{**case, "softcap": 1e-46}, stream=0)
    assert e.value.status == SHAPE
