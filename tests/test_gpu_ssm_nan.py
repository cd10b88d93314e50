"""NaN in the scan's parameters: every variant lets it through to its channel and its state, and to no other."""

import numpy as np
import pytest
import torch

from block_cases import offsets, scan_inputs
from ssm_compressed_chunked_b200 import attamba as A
from test_gpu_ssm_block import run_scan

pytestmark = pytest.mark.gpu


# eight lanes a channel; four; two; one (2^27 tokens x channels x states or more: the first of every 8 state pairs has its
# decay on the FMA pipe)
@pytest.mark.parametrize("dtype,D,N,T", [(torch.float32, 64, 16, 40), (torch.bfloat16, 64, 32, 900), (torch.bfloat16, 512, 16, 1200),
                                         (torch.bfloat16, 2048, 16, 4100), (torch.float32, 1024, 32, 4100)])
def test_nan_in_a_reaches_its_channel(dtype, D, N, T):
    lens = [T // 3, 0, T // 2]
    n, cu = sum(lens), offsets(lens)
    d = scan_inputs(T, D, N, dtype, seed=D + N)
    state = torch.randn(3, N, D, generator=torch.Generator().manual_seed(1))
    clean, cst, status = run_scan(d, cu, T, dtype, state, None, [1, 1, 0])
    bad = {0: 0, 7: 1, 33: N // 2, D - 1: N - 1}         # channel: the state whose A is NaN
    dirty = dict(d, A=d["A"].clone())
    for c, s in bad.items():
        dirty["A"][c, s] = float("nan")
    y, st, status2 = run_scan(dirty, cu, T, dtype, state, None, [1, 1, 0])
    assert status == 0 and status2 == 0
    good = [c for c in range(D) if c not in bad]
    assert torch.equal(y[:n][:, good], clean[:n][:, good])
    assert torch.equal(st[:, :, good], cst[:, :, good])
    for c, s in bad.items():
        assert bool(torch.isnan(y[:n, c]).all()), c
        for seq in (0, 2):
            isnan = torch.isnan(st[seq, :, c]).cpu().numpy()
            assert np.array_equal(np.flatnonzero(isnan), [s]), (c, seq)
        rest = [k for k in range(N) if k != s]
        assert torch.equal(st[:, rest, c], cst[:, rest, c])
        assert torch.equal(st[1, :, c], state[1, :, c].cuda())      # an empty sequence's state stays as it was
