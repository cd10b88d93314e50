"""The text of an AttambaError is the refused call's own (no GPU needed)."""

import ctypes

import pytest

from ssm_compressed_chunked_b200 import attamba as A

FAKE = 1 << 20


def refuse_a_convolution():
    st = A.load().attamba_causal_conv(A.BF16, FAKE, 64, FAKE, None, 64, 9, A.ACT_SILU,
                                      ctypes.byref(A.SeqsT(FAKE, None, None, 4, 1)), None, 0, FAKE, 64, None, None)
    with pytest.raises(A.AttambaError, match=r"^attamba_causal_conv: unsupported shape or dtype attamba_causal_conv: K is 2, 3 or 4$"):
        A._check(st, "attamba_causal_conv")


def test_a_refusal_without_a_reason_borrows_none():
    """The older entry points refuse most bad arguments without a reason of their own: the thread's error text is then the
    last other refusal's, and says nothing about this call."""
    L = A.load()
    idx = A.IndexT(FAKE, FAKE, FAKE, FAKE, FAKE, 4, 1, 16)
    calls = {
        "attamba_chunk_index": lambda: L.attamba_chunk_index(None, 4, 1, 16, 4, 0, 0, 7, ctypes.byref(idx), None, None),
        "attamba_kv_ssm_scan": lambda: L.attamba_kv_ssm_scan(1, *([FAKE] * 12), 4, 16, 64, 24, FAKE, FAKE, None, None, None, None),
        "attamba_proj_gemm": lambda: L.attamba_proj_gemm(A.BF16, FAKE, FAKE, 0, 64, 64, None, 0, None, None),
        "attamba_selftest_wait_timeout": lambda: L.attamba_selftest_wait_timeout(999, FAKE, None)}
    for name, call in calls.items():
        refuse_a_convolution()
        with pytest.raises(A.AttambaError) as e:
            A._check(call(), name)
        assert str(e.value).startswith(name + ": ") and "attamba_causal_conv" not in str(e.value), str(e.value)


def test_a_refusal_with_a_reason_keeps_it():
    L = A.load()
    c = A.CacheT(*([FAKE] * 8), 1, 1, 64, 16, 8, 0, 4, 3)
    refuse_a_convolution()
    with pytest.raises(A.AttambaError, match="attamba_cache_from_prefill: invalid argument attamba_cache_from_prefill: .* exceed cap 3"):
        A._check(L.attamba_cache_from_prefill(1, ctypes.byref(c), *([FAKE] * 13), 64, None, None), "attamba_cache_from_prefill")
    refuse_a_convolution()
