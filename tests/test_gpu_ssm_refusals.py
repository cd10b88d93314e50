"""Calls of the SSM block's operators that the binding refuses for what only a CUDA tensor can show."""

import pytest
import torch

from ssm_compressed_chunked_b200 import attamba as A
from test_gpu_ssm_block import i32

pytestmark = pytest.mark.gpu


def test_a_state_without_slots_is_refused():
    """An empty state has a null address, which the C ABI takes for no state: the call would run and keep nothing."""
    D, N, K, T = 64, 16, 4, 5
    f32 = torch.float32
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    x, y, w, a, b = z(T, D), z(T, D), z(D, K, dt=f32), -torch.ones(D, N, device="cuda"), z(T, N)
    seqs = A.Seqs(i32([0, T]), T, slots=i32([0]), cont=i32([1]))
    win, st = z(0, K - 1, D), z(0, N, D, dt=f32)
    for call in (lambda: A.causal_conv(x, w, None, seqs, y, state=win), lambda: A.conv_step(x, w, None, win, y),
                 lambda: A.selective_scan(x, x, None, a, b, b, seqs, y, state=st),
                 lambda: A.scan_step(x, x, None, a, b, b, st, y)):
        with pytest.raises(A.AttambaError, match="state has no slots"):
            call()
    A.causal_conv(x, w, None, seqs, y)                 # no state at all stays allowed
    A.selective_scan(x, x, None, a, b, b, seqs, y)
