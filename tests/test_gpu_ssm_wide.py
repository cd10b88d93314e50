"""The SSM block's operators at width: element offsets past 2^31 (token rows 65536 bytes apart, states of more than 2^31
elements; the rows past the border are compared with the oracle, which sees the same tokens next to each other), the scan's
variants for long and wide batches on sampled channels, and two streams on one state array."""

import numpy as np
import pytest
import torch

from block_cases import HALF, TINY, U, assert_within, offsets, scan_bound, scan_inputs
from helpers import f64
from oracle import block as OB
from ssm_compressed_chunked_b200 import attamba as A
from test_gpu_ssm_block import conv_bound, i32, new_status, run_scan, workspace

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
STRIDE, T = 32768, 65800          # T * STRIDE = 2^31 + 8.6e6 elements
KEPT = 600                        # the rows that are compared: the last ones, most of them past the border


@pytest.fixture(scope="module")
def wide():
    """Two arrays [T, STRIDE]: inputs and outputs, touched in a few columns only."""
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    arrays = [torch.empty(T, STRIDE, dtype=BF, device="cuda") for _ in range(2)]
    yield arrays
    del arrays
    torch.cuda.empty_cache()


def place(buf, col, t):
    w = buf[:, col:col + t.shape[1]]
    w.copy_(t)
    return w


def test_rows_past_2_31_elements(wide):
    D, N, K = 8, 16, 4
    inp, out = wide
    d = scan_inputs(T, D, N, BF, seed=1)
    cols, at = {}, STRIDE - 128                     # the last columns of the array
    for k in ("x", "dt", "z", "B", "C"):
        cols[k] = place(inp, at, d[k].cuda())
        at += d[k].shape[1]
    lens = [T - KEPT, 0, 40, KEPT - 43]             # the last sequences lie in the compared rows; three rows behind them
    cu = offsets(lens)
    seqs, status = A.Seqs(i32(cu), T), new_status()
    y, cy = out[:, STRIDE - 8:], out[:, STRIDE - 16:STRIDE - 8]
    out[:, STRIDE - 16:].fill_(float("nan"))
    st = torch.zeros(4, N, D, device="cuda")
    A.selective_scan(cols["x"], cols["dt"], d["bias"].cuda(), d["A"].cuda(), cols["B"], cols["C"], seqs, y,
                     skip=d["skip"].cuda(), z=cols["z"], state=st, workspace=workspace(T, D, N), status=status)
    w = torch.randn(D, K, generator=torch.Generator().manual_seed(2))
    win = torch.zeros(4, K - 1, D, dtype=BF, device="cuda")
    A.causal_conv(cols["x"], w.cuda(), None, seqs, cy, state=win, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    tail = slice(T - KEPT, T)
    part = {k: (v[tail] if k in ("x", "dt", "z", "B", "C") else v) for k, v in d.items()}
    n = {k: f64(v) for k, v in part.items()}
    sub = offsets(lens[1:])
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], sub, n["skip"], n["z"],
                                    np.zeros((3, N, D)))
    by, bst = scan_bound(part, sub, BF, torch.zeros(3, N, D))
    m = KEPT - 3
    assert_within(f64(y[tail])[:m], ref[:m], by[:m], "scan y")
    assert_within(f64(st)[1:], ref_st, bst, "scan state")
    pre, _ = OB.causal_conv(n["x"], f64(w), None, sub, act="linear")
    ref, ref_win = OB.causal_conv(n["x"], f64(w), None, sub, np.zeros((3, K - 1, D)))
    assert_within(f64(cy[tail])[:m], ref[:m], conv_bound(part["x"], w, None, pre, ref, sub, BF, "silu")[:m], "conv y")
    assert np.array_equal(f64(win)[1:], ref_win)
    assert bool(torch.isnan(out[T - 3:, STRIDE - 16:]).all())
    # the norm over the same rows
    g = torch.rand(D, generator=torch.Generator().manual_seed(3)) + 0.5
    r, h = out[:, :8], out[:, 8:16]
    A.block_norm(cols["x"], cols["dt"], r, h, w_post=g.cuda(), w_pre=g.cuda(), gate=cols["z"], alpha=0.5)
    rr, hh = OB.block_norm(n["x"], n["dt"], w_post=f64(g), w_pre=f64(g), gate=n["z"], alpha=0.5)
    # bf16's half step, and fp32's few dozen steps on values of order 1 (gate, root, three products): under 2^-17
    bound = lambda v: (HALF[BF] + 2.0 ** -17) * np.abs(v) + 2.0 ** -17 + TINY  # noqa: E731
    assert_within(f64(r[tail]), rr, bound(rr), "norm r")
    assert_within(f64(h[tail]), hh, bound(hh) + 60 * U, "norm h")


def test_states_past_2_31_elements():
    """Slots at both ends of a state of 2^31 + 2^26 elements, for a prompt and for single tokens."""
    D, N, K = 4096, 16, 4
    n_slots = (2 ** 31 + 2 ** 26) // (N * D)
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    st = torch.zeros(n_slots, N, D, device="cuda")
    slots = [n_slots - 1, 0, n_slots - 2]
    d = scan_inputs(3, D, N, BF, seed=4)
    g = {k: v.cuda() for k, v in d.items()}
    init = torch.randn(3, N, D, generator=torch.Generator().manual_seed(5))
    st[slots] = init.cuda()
    y, status = torch.zeros(3, D, dtype=BF, device="cuda"), new_status()
    A.scan_step(g["x"], g["dt"], g["bias"], g["A"], g["B"], g["C"], st, y, skip=g["skip"], z=g["z"], slots=i32(slots),
                status=status)
    n = {k: f64(v) for k, v in d.items()}
    cu, cont = offsets([1, 1, 1]), [1, 1, 1]
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], cu, n["skip"], n["z"], f64(init),
                                    None, cont)
    by, bst = scan_bound(d, cu, BF, init, None, cont)
    assert_within(f64(y), ref, by, "step y")
    assert_within(f64(st[slots]), ref_st, bst, "step state")
    st[slots] = init.cuda()
    y.zero_()
    A.selective_scan(g["x"], g["dt"], g["bias"], g["A"], g["B"], g["C"], A.Seqs(i32(cu), 3, slots=i32(slots), cont=i32(cont)),
                     y, skip=g["skip"], z=g["z"], state=st, status=status)
    assert_within(f64(y), ref, by, "prompt y")
    assert_within(f64(st[slots]), ref_st, bst, "prompt state")
    assert status.item() == 0 and float(st[n_slots // 2].abs().max()) == 0.0
    del st
    torch.cuda.empty_cache()


def channels_of(d, pick):
    """The scan's inputs restricted to some channels (they do not mix; B and C are shared)."""
    cut = lambda k, v: None if v is None else v[:, pick] if k in ("x", "dt", "z") else v[pick] if k in ("A", "bias", "skip") else v  # noqa: E731
    return {k: cut(k, v) for k, v in d.items()}


# one lane a channel from 2^27 tokens x channels x states on, two below, four for narrow blocks; ragged sequences that end inside
# and on tiles' ends, empty ones, kept and fresh states
@pytest.mark.parametrize("dtype,D,N,lens,pad", [("bf16", 2048, 16, [1500, 0, 37, 2000, 1, 600], 5), ("f32", 2048, 16, [4100], 0),
                                                ("bf16", 2048, 32, [700, 1399], 3), ("f32", 1024, 32, [4096], 0),
                                                ("bf16", 512, 16, [300, 0, 1, 512, 77], 9), ("f32", 512, 32, [130, 500], 0),
                                                ("bf16", 1024, 16, [2048], 0), ("f32", 2056, 16, [129], 2)])
def test_scan_variants_on_sampled_channels(dtype, D, N, lens, pad):
    dt = {"bf16": BF, "f32": torch.float32}[dtype]
    T, S = sum(lens) + pad, len(lens)
    d = scan_inputs(T, D, N, dt, seed=D + N + S)
    cu = offsets(lens)
    rng = np.random.default_rng(S)
    slots, cont = rng.permutation(S + 2)[:S], rng.integers(0, 2, S)
    state = torch.randn(S + 2, N, D, generator=torch.Generator().manual_seed(S))
    y, st, status = run_scan(d, cu, T, dt, state, slots, cont)
    assert status == 0
    pick = sorted({0, 1, 31, 32, 127, 128, 255, 256, D // 2 - 1, D // 2, D - 2, D - 1})
    part = channels_of(d, pick)
    n = {k: f64(v) for k, v in part.items()}
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], cu, n["skip"], n["z"],
                                    f64(state[:, :, pick]), slots, cont)
    by, bst = scan_bound(part, cu, dt, state[:, :, pick], slots, cont)
    m = sum(lens)
    assert bool(torch.isnan(y[m:]).all()) and not bool(torch.isnan(y[:m]).any())
    assert_within(f64(y[:m][:, pick]), ref[:m], by[:m], "y")
    assert_within(f64(st[:, :, pick])[slots], ref_st[slots], bst[slots], "state")


def test_two_streams_share_a_state_array():
    """Prompts and steps of disjoint slots of one state array on two streams at once, a workspace each, against the same
    calls one after the other."""
    D, N, T = 512, 16, 500
    both = [scan_inputs(T, D, N, BF, seed=60 + k) for k in range(2)]
    g = [{k: v.cuda() for k, v in d.items()} for d in both]
    start = torch.randn(8, N, D, generator=torch.Generator().manual_seed(7)).cuda()
    slots = [i32([0, 2, 4, 6]), i32([7, 5, 3, 1])]
    seqs = [A.Seqs(i32([0, 100, 100, 333, 500]), T, slots=s, cont=i32([1, 0, 1, 1])) for s in slots]
    ws = [workspace(T, D, N) for _ in range(2)]

    def calls(k, st, out):
        a = g[k]
        for _ in range(10):
            A.selective_scan(a["x"], a["dt"], a["bias"], a["A"], a["B"], a["C"], seqs[k], out, skip=a["skip"], z=a["z"],
                             state=st, workspace=ws[k])
            A.scan_step(a["x"][:4], a["dt"][:4], a["bias"], a["A"], a["B"][:4], a["C"][:4], st, out[:4], slots=slots[k])

    st1, out1 = start.clone(), [torch.zeros(T, D, dtype=BF, device="cuda") for _ in range(2)]
    for k in range(2):
        calls(k, st1, out1[k])
    st2, out2 = start.clone(), [torch.zeros(T, D, dtype=BF, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            calls(k, st2, out2[k])
    torch.cuda.synchronize()
    assert torch.equal(st1, st2) and all(torch.equal(a, b) for a, b in zip(out1, out2))
