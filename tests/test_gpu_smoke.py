"""The smoke entry point runs every family of calls on the GPU."""
import pytest

import __graft_entry__
from attention_forward_sm_gb300 import binding as attn

pytestmark = pytest.mark.gpu


def test_smoke_calls_every_family(monkeypatch):
    lib, called = attn.load(), set()

    class Counting:
        def __getattr__(self, name):
            called.add(name)
            return getattr(lib, name)

    monkeypatch.setattr(attn, "_lib", Counting())
    __graft_entry__.smoke()
    assert {"attn_fwd", "attn_decode_splitkv", "attn_fwd_mod", "attn_row_ranges", "attn_decode_varlen",
            "attn_decode_prefix"} <= called
