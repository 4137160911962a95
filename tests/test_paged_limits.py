"""Limits of the attention calls over a paged cache that belong to one of its kernels: no GPU is
needed to see that a call gets past the checks of its sizes."""
import pytest
import torch

from attention_forward_sm_gb300 import binding as attn
from test_paged_abi import A, FWD, NULL, SHAPE, lib  # noqa: F401

# rows and a table within a table of 2^18 tokens, whose units of work would not fit 32 bits
LARGE = [dict(B=1, T=131072, max_new=131072, Hq=64, Hkv=8, q_stride=8192, D=128, page=128, M=1024),
         dict(B=4, T=65536, max_new=65536, Hq=64, Hkv=8, q_stride=4096, page=16, M=2**14),
         dict(B=1, T=2**24, max_new=3, Hq=128, Hkv=8, q_stride=8192, page=64, M=2**12)]


@pytest.mark.parametrize("change", LARGE)
def test_many_rows_have_no_limit_of_units(lib, change):  # noqa: F811
    case = {**FWD, **change}
    assert lib.attn_paged_fwd(*{**case, "lse": 0}.values(), None) == NULL
    if not torch.cuda.is_available():  # (the addresses are not anyone's)
        assert lib.attn_paged_fwd(*case.values(), None) not in (0, SHAPE)


@pytest.mark.parametrize("change", [dict(max_new=1, Hq=16, q_stride=1024), dict(M=2**14 + 1)])
def test_few_rows_have_one(lib, change):  # noqa: F811
    case = {**FWD, **LARGE[1], **change}
    assert lib.attn_paged_fwd(*{**case, "T": 2**24}.values(), None) == SHAPE


@pytest.mark.gpu
def test_a_large_batch_of_rows_runs():
    """What the first of these asks for, most rows nobody's."""
    import paged_ref as ref
    from test_gpu_paged import check_attention
    c = ref.Cache([400], 8, 64, 128, False, seed=1)
    table = torch.full((1, 1024), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    q = torch.zeros(131072, 64, 64, dtype=torch.bfloat16, device="cuda")
    q[:70] = torch.randn(70, 64, 64, device="cuda")
    offsets = ref.offsets_of([70])
    o, lse = attn.paged_forward(q, c.kp, c.vp, table, c.lens_t, offsets)
    check_attention(o[:70], lse[:70], q[:70], c, offsets)
