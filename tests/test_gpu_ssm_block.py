"""The SSM block's operators on the GPU against the float64 oracle: short convolution, selective scan, their
single-token steps, and the block norm.  Outputs are poisoned first and lie between guards; carried states too."""

import numpy as np
import pytest
import torch

from block_cases import (DT, HALF, TINY, U, act_bound, assert_within, offsets, scan_bound, scan_inputs, to_gpu, wide)
from helpers import Guarded, f64
from oracle import block as OB
from ssm_compressed_chunked_b200 import attamba as A

pytestmark = pytest.mark.gpu


def i32(v):
    return None if v is None else torch.tensor(np.asarray(v, dtype=np.int32)).cuda()


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def guarded_copy(guard, t):
    g = guard(tuple(t.shape), t.dtype)
    g.copy_(t)
    return g


def workspace(T, D, N):
    n = A.selective_scan_workspace_size(T, D, N)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None      # NaN: nothing may count on it


def assert_tail_untouched(y, total, what):
    """Rows no sequence owns still hold the canary (NaN)."""
    assert bool(torch.isnan(y[total:]).all()), f"{what}: rows behind the last sequence were written"


# ---------------------------------------------------------------- convolution
LENS = [[1], [2], [3], [61], [16, 16, 16, 16], [0, 5, 0, 0, 17, 3, 1, 2, 64, 16, 15, 33, 0], [15, 1, 1, 1, 47, 200, 1, 0],
        [0], [513], [1] * 70]


def conv_bound(x, w, bias, ref_pre, ref, cu, dtype, act, state=None, slots=None, cont=None):
    """n u of the magnitudes (bias, K products), SiLU's slope of at most 1.1, the quotient, the stored rounding."""
    mag, _ = OB.causal_conv(np.abs(f64(x)), np.abs(f64(w)), None if bias is None else np.abs(f64(bias)), cu,
                            None if state is None else np.abs(f64(state)), slots, cont, act="linear")
    K = w.shape[1]
    b = 1.1 * (K + 2) * U * mag
    if act == "silu":
        b = b + np.abs(ref) * act_bound("silu", ref_pre)
    return b + HALF[dtype] * (np.abs(ref) + b) + TINY


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("dtype,D,K", [("bf16", 264, 4), ("f32", 136, 3), ("bf16", 8, 2), ("f32", 8, 4), ("bf16", 520, 3)])
def test_conv(lens, dtype, D, K):
    lens = LENS[lens]
    S, total = len(lens), sum(lens)
    T = max(1, total + (S % 3) * 9)
    g = torch.Generator().manual_seed(S * 100 + D + K)
    dt = DT[dtype]
    x = wide(T, D, dt, g, extra=16 if K == 3 else 0)
    w, bias = torch.randn(D, K, generator=g) / K, torch.randn(D, generator=g) if K != 3 else None
    act = "silu" if K != 2 else "linear"
    cu = offsets(lens)
    slots = np.random.default_rng(S).permutation(S + 4)[:S]
    if S > 2:
        slots[1] = -1
    cont = np.random.default_rng(S + 1).integers(0, 2, S)
    state = torch.randn(S + 4, K - 1, D, generator=g).to(dt)
    guard = Guarded()
    st = guarded_copy(guard, state)
    y, status = guard((T, D), dt), new_status()
    seqs = A.Seqs(i32(cu), T, slots=i32(slots), cont=i32(cont))
    A.causal_conv(to_gpu(x), w.cuda(), to_gpu(bias), seqs, y, state=st, act=A.ACT_SILU if act == "silu" else A.ACT_LINEAR,
                  status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    guard.check()
    args = (f64(x), f64(w), None if bias is None else f64(bias), cu, f64(state), slots, cont)
    pre, _ = OB.causal_conv(*args, act="linear")
    ref, ref_st = OB.causal_conv(*args, act=act)
    assert_tail_untouched(y, total, "conv")
    assert_within(f64(y)[:total], ref[:total],
                  conv_bound(x, w, bias, pre, ref, cu, dt, act, state, slots, cont)[:total], "conv y")
    assert np.array_equal(f64(st), ref_st), "the carried window holds copies of inputs: exact"


@pytest.mark.parametrize("with_state", [True, False])
def test_conv_without_slots_or_flags(with_state):
    """No slot map: sequence s has state row s; no flags: none continues, rows are written; no state: none at all."""
    lens, D, K = [9, 30, 4], 64, 4
    g = torch.Generator().manual_seed(7)
    x, w = wide(43, D, torch.float32, g), torch.randn(D, K, generator=g)
    state = torch.randn(3, K - 1, D, generator=g)
    st, y, status = state.cuda(), torch.zeros(43, D, device="cuda"), new_status()
    A.causal_conv(x.cuda(), w.cuda(), None, A.Seqs(i32(offsets(lens)), 43), y, state=st if with_state else None, status=status)
    ref, ref_st = OB.causal_conv(f64(x), f64(w), None, offsets(lens), f64(state))
    pre, _ = OB.causal_conv(f64(x), f64(w), None, offsets(lens), act="linear")
    assert_within(f64(y), ref, conv_bound(x, w, None, pre, ref, offsets(lens), torch.float32, "silu"), "conv")
    assert np.array_equal(f64(st), ref_st if with_state else f64(state)) and status.item() == 0


@pytest.mark.parametrize("dtype,B,D,K", [("bf16", 1, 264, 4), ("f32", 5, 136, 3), ("bf16", 130, 72, 2), ("f32", 33, 8, 4)])
def test_conv_step(dtype, B, D, K):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(B + D)
    x, w, bias = wide(B, D, dt, g, extra=8), torch.randn(D, K, generator=g), torch.randn(D, generator=g)
    state = torch.randn(B + 3, K - 1, D, generator=g).to(dt)
    slots = np.random.default_rng(B).permutation(B + 3)[:B]
    if B > 4:
        slots[[2, B - 1]] = -1
    guard = Guarded()
    st, y, status = guarded_copy(guard, state), guard((B, D), dt), new_status()
    A.conv_step(to_gpu(x), w.cuda(), bias.cuda(), st, y, slots=i32(slots), status=status)
    torch.cuda.synchronize()
    guard.check()
    assert status.item() == 0
    cu, cont = offsets([1] * B), np.ones(B, dtype=int)
    args = (f64(x), f64(w), f64(bias), cu, f64(state), slots, cont)
    pre, _ = OB.causal_conv(*args, act="linear")
    ref, ref_st = OB.causal_conv(*args)
    live = slots >= 0
    assert bool(torch.isnan(y[torch.from_numpy(~live).cuda()]).all())
    b = conv_bound(x, w, bias, pre, ref, cu, dt, "silu", state, slots, cont)
    assert_within(f64(y)[live], ref[live], b[live], "conv_step y")
    assert np.array_equal(f64(st), ref_st)


# ---------------------------------------------------------------- scan
def run_scan(d, cu, T, dtype, state=None, slots=None, cont=None):
    guard = Guarded()
    D, N = d["A"].shape
    st = None if state is None else guarded_copy(guard, state)
    y, status = guard((T, D), dtype), new_status()
    seqs = A.Seqs(i32(cu), T, slots=i32(slots), cont=i32(cont))
    A.selective_scan(*(to_gpu(d[k]) for k in ("x", "dt", "bias", "A", "B", "C")), seqs, y, skip=to_gpu(d["skip"]),
                     z=to_gpu(d["z"]), state=st, workspace=workspace(T, D, N), status=status)
    torch.cuda.synchronize()
    guard.check()
    return y, st, status.item()


SCAN_LENS = [[1], [2], [0], [61], [128], [129], [127, 1, 128], [0, 5, 0, 300, 3, 1, 2, 64, 0, 15, 133, 0], [1] * 40, [513],
             [700, 1]]


@pytest.mark.parametrize("lens", range(len(SCAN_LENS)))
@pytest.mark.parametrize("dtype,D,N,full", [("bf16", 72, 16, True), ("f32", 264, 16, True), ("bf16", 136, 32, True),
                                            ("f32", 8, 32, False), ("f32", 72, 16, False)])
def test_scan(lens, dtype, D, N, full):
    lens = SCAN_LENS[lens]
    S, total = len(lens), sum(lens)
    T = max(1, total + (S % 3) * 13)
    dt = DT[dtype]
    d = scan_inputs(T, D, N, dt, seed=S * 7 + D, gate=full, skip=full, bias=full, extra=16 if full else 0)
    cu = offsets(lens)
    slots = np.random.default_rng(S).permutation(S + 4)[:S]
    if S > 2:
        slots[1] = -1
    cont = np.random.default_rng(S + 1).integers(0, 2, S)
    state = torch.randn(S + 4, N, D, generator=torch.Generator().manual_seed(S))
    y, st, status = run_scan(d, cu, T, dt, state, slots, cont)
    assert status == 0
    n = {k: (None if v is None else f64(v)) for k, v in d.items()}
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], cu, n["skip"], n["z"], f64(state),
                                    slots, cont)
    by, bst = scan_bound(d, cu, dt, state, slots, cont)
    assert_tail_untouched(y, total, "scan")
    assert_within(f64(y)[:total], ref[:total], by[:total], "scan y")
    used = [int(s) for s in slots if s >= 0]
    assert_within(f64(st)[used], ref_st[used], bst[used], "scan state")
    rest = [r for r in range(S + 4) if r not in used]
    assert torch.equal(st.cpu()[rest], state[rest]), "rows of no sequence stay as they were"


def test_scan_without_state_and_the_tail_of_long_memory():
    """No state at all, and decays so near 1 that the first tokens still count at the end: the tiles are joined."""
    T, D, N = 1000, 64, 16
    d = scan_inputs(T, D, N, torch.float32, seed=5)
    d["bias"] = torch.full((D,), -9.0)
    d["dt"] = d["dt"] * 0.1
    d["A"] = d["A"] / 16
    cu = offsets([T])
    y, _, status = run_scan(d, cu, T, torch.float32)
    n = {k: f64(v) for k, v in d.items()}
    ref, _ = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], cu, n["skip"], n["z"])
    by, _ = scan_bound(d, cu, torch.float32)
    assert status == 0
    assert_within(f64(y), ref, by, "scan y")


def test_scan_in_pieces_equals_the_whole():
    """A prompt in three calls, each continuing from the state row, against the prompt in one call."""
    T, D, N = 420, 136, 16
    d = scan_inputs(T, D, N, torch.float32, seed=3)
    state = torch.randn(2, N, D, generator=torch.Generator().manual_seed(1))
    whole, wst, _ = run_scan(d, offsets([T]), T, torch.float32, state, [1], [0])
    st = state
    rows = []
    for a, b, cont in ((0, 130, 0), (130, 131, 1), (131, T, 1)):
        part = {k: (v[a:b].contiguous() if k in ("x", "dt", "B", "C", "z") else v) for k, v in d.items()}
        y, st, status = run_scan(part, offsets([b - a]), b - a, torch.float32, st.cpu(), [1], [cont])
        assert status == 0
        rows.append(y)
    by, bst = scan_bound(d, offsets([T]), torch.float32, state, [1], [0])
    assert_within(f64(torch.cat(rows)), f64(whole), 2 * by, "pieces y")
    assert_within(f64(st)[1], f64(wst)[1], 2 * bst[1], "pieces state")


@pytest.mark.parametrize("dtype,B,D,N,full", [("bf16", 1, 264, 16, True), ("f32", 7, 136, 32, True), ("bf16", 70, 72, 32, False),
                                              ("f32", 33, 8, 16, False), ("bf16", 3, 1032, 16, True)])
def test_scan_step(dtype, B, D, N, full):
    dt = DT[dtype]
    d = scan_inputs(B, D, N, dt, seed=B + D, gate=full, skip=full, bias=full, extra=8 if full else 0)
    state = torch.randn(B + 3, N, D, generator=torch.Generator().manual_seed(B))
    slots = np.random.default_rng(B).permutation(B + 3)[:B]
    if B > 4:
        slots[[2, B - 1]] = -1
    guard = Guarded()
    st, y, status = guarded_copy(guard, state), guard((B, D), dt), new_status()
    A.scan_step(*(to_gpu(d[k]) for k in ("x", "dt", "bias", "A", "B", "C")), st, y, skip=to_gpu(d["skip"]),
                z=to_gpu(d["z"]), slots=i32(slots), status=status)
    torch.cuda.synchronize()
    guard.check()
    assert status.item() == 0
    cu, cont = offsets([1] * B), np.ones(B, dtype=int)
    n = {k: (None if v is None else f64(v)) for k, v in d.items()}
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], cu, n["skip"], n["z"], f64(state),
                                    slots, cont)
    by, bst = scan_bound(d, cu, dt, state, slots, cont)
    live = slots >= 0
    assert bool(torch.isnan(y[torch.from_numpy(~live).cuda()]).all())
    assert_within(f64(y)[live], ref[live], by[live], "scan_step y")
    used = slots[live]
    assert_within(f64(st)[used], ref_st[used], bst[used], "scan_step state")
    rest = [r for r in range(B + 3) if r not in used]
    assert torch.equal(st.cpu()[rest], state[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_steps(dtype):
    """delta from 0 (dt very negative: the state stays) to huge (the state is replaced); closed gates."""
    D, N, T = 64, 16, 40
    dt = DT[dtype]
    d = scan_inputs(T, D, N, dt, seed=11)
    v = torch.tensor([-200.0, -90.0, -30.0, -1.0, 0.0, 19.0, 21.0, 80.0, 1000.0])
    d["dt"] = v.repeat(T * D // 9 + 1)[:T * D].reshape(T, D).to(dt)
    d["z"] = torch.tensor([-200.0, -88.0, -20.0, 0.0, 30.0, 100.0, 1.0]).repeat(T * D // 7 + 1)[:T * D].reshape(T, D).to(dt)
    state = torch.randn(1, N, D, generator=torch.Generator().manual_seed(2))
    y, st, status = run_scan(d, offsets([T]), T, dt, state, None, [1])
    n = {k: f64(t) for k, t in d.items()}
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], offsets([T]), n["skip"], n["z"],
                                    f64(state), None, [1])
    by, bst = scan_bound(d, offsets([T]), dt, state, None, [1])
    assert status == 0
    assert_within(f64(y), ref, by, "y")
    assert_within(f64(st), ref_st, bst, "state")


# ---------------------------------------------------------------- both
def test_not_a_number_stays_in_its_sequence():
    """NaN and infinities in one sequence, in its carried state and behind the last one reach no other: the others'
    outputs and states are bit for bit those of a clean batch."""
    lens, D, N, K, T = [140, 150, 0, 137], 64, 16, 4, 440
    d = scan_inputs(T, D, N, torch.float32, seed=21)
    state = torch.randn(4, N, D, generator=torch.Generator().manual_seed(4))
    cu, cont = offsets(lens), [1, 1, 1, 1]
    clean, cst, _ = run_scan(d, cu, T, torch.float32, state, None, cont)
    dirty = {k: (None if v is None else v.clone()) for k, v in d.items()}
    for k, bad in (("x", float("nan")), ("dt", float("inf")), ("B", float("inf")), ("C", float("nan")), ("z", float("-inf"))):
        dirty[k][145:290] = bad
        dirty[k][427:] = bad
    bad_state = state.clone()
    bad_state[1] = float("nan")
    y, st, status = run_scan(dirty, cu, T, torch.float32, bad_state, None, cont)
    assert status == 0
    for a, b in ((0, 140), (290, 427)):
        assert torch.equal(y[a:b], clean[a:b])
    assert torch.equal(st[[0, 2, 3]], cst[[0, 2, 3]])
    w = torch.randn(D, K, generator=torch.Generator().manual_seed(5)).cuda()
    out = []
    for src in (d, dirty):
        win = torch.ones(4, K - 1, D, device="cuda")
        win[1] = float("nan") if src is dirty else 1.0
        yy = torch.zeros(T, D, device="cuda")
        A.causal_conv(src["x"].cuda(), w, None, A.Seqs(i32(cu), T, cont=i32(cont)), yy, state=win)
        out.append((yy, win))
    for a, b in ((0, 140), (290, 427)):
        assert torch.equal(out[0][0][a:b], out[1][0][a:b])
    assert torch.equal(out[0][1][[0, 2, 3]], out[1][1][[0, 2, 3]])


def test_repeated_and_wrong_slots_are_reported_and_keep_nothing():
    """One slot named twice, or out of range: the status bit, the first one's state, no other row touched."""
    D, N, K = 64, 16, 3
    d = scan_inputs(12, D, N, torch.float32, seed=31)
    state = torch.randn(4, N, D, generator=torch.Generator().manual_seed(6))
    for slots, first in (([2, 2, 0], True), ([1, 7, 0], False), ([1, -5, 0], False)):
        y, st, status = run_scan(d, offsets([4, 5, 3]), 12, torch.float32, state, slots, [1, 1, 1])
        good, gst, ok = run_scan(d, offsets([4, 5, 3]), 12, torch.float32, state, [slots[0], -1, 0], [1, 1, 1])
        assert status == A.DEV_BAD_SEQS and ok == 0
        assert torch.equal(y, good) and torch.equal(st, gst)
        rows = {k: d[k][:3].cuda() for k in ("x", "dt", "B", "C", "z")}
        outs = []
        for sl in (slots, [slots[0], -1, 0]):
            s2, yy, flag = state.cuda(), torch.zeros(3, D, device="cuda"), new_status()
            A.scan_step(rows["x"], rows["dt"], d["bias"].cuda(), d["A"].cuda(), rows["B"], rows["C"], s2, yy, slots=i32(sl),
                        status=flag)
            c2 = torch.ones(4, K - 1, D, device="cuda")
            cy = torch.zeros(3, D, device="cuda")
            A.conv_step(rows["x"], torch.ones(D, K, device="cuda"), None, c2, cy, slots=i32(sl), status=flag)
            outs.append((s2, yy, c2, cy, flag.item()))
        assert outs[0][4] == A.DEV_BAD_SEQS and outs[1][4] == 0
        assert all(torch.equal(a, b) for a, b in zip(outs[0][:4], outs[1][:4]))


@pytest.mark.parametrize("cu", [[0, 9, 5, 12], [0, 4, 900, 12], [3, 4, 8, 12], [0, 4, 8, 400], [-7, 4, 8, 12], [0, 2 ** 31 - 1, 8, 12],
                                [12, 8, 4, 0], [0, -2 ** 31, -5, -1]])
def test_malformed_offsets_are_reported_and_stay_inside(cu):
    """Offsets that decrease, start late or end behind T raise the status bit; nothing outside the arrays is written."""
    T, D, N, K = 300, 64, 16, 4
    d = scan_inputs(T, D, N, torch.float32, seed=41)
    guard = Guarded()
    st = guarded_copy(guard, torch.zeros(3, N, D))
    y, win, cy = guard((T, D), torch.float32), guarded_copy(guard, torch.zeros(3, K - 1, D)), guard((T, D), torch.float32)
    seqs, one, two = A.Seqs(i32(cu), T), new_status(), new_status()
    size = A.selective_scan_workspace_size(T, D, N)
    ws = guard((max(size, 4) // 4,), torch.float32)
    A.selective_scan(*(to_gpu(d[k]) for k in ("x", "dt", "bias", "A", "B", "C")), seqs, y, state=st, workspace=ws, status=one)
    A.causal_conv(d["x"].cuda(), torch.ones(D, K, device="cuda"), None, seqs, cy, state=win, status=two)
    torch.cuda.synchronize()
    guard.check()
    assert one.item() == A.DEV_BAD_SEQS and two.item() == A.DEV_BAD_SEQS


def test_the_binding_checks_types_shapes_strides_and_devices():
    D, N, K = 64, 16, 4
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    f32 = torch.float32
    ok = dict(x=z(4, D), w=z(D, K, dt=f32), bias=z(D, dt=f32), state=z(5, K - 1, D), y=z(4, D), slots=i32([0, 1, 2, 3]))
    A.conv_step(**ok)
    wide = z(4, 2 * D)
    for key, bad in (("x", z(4, D, 1)), ("x", z(0, D)), ("x", z(4, D, dt=torch.float16)), ("x", z(4, D).cpu()), ("y", z(3, D)),
                     ("y", z(4, D, dt=f32)), ("y", z(D, 4).t()), ("y", z(4, D).cpu()), ("w", z(D, K)), ("w", z(K, D, dt=f32).t()),
                     ("w", z(D, K, dt=f32).cpu()), ("bias", z(D + 8, dt=f32)), ("bias", z(2 * D, dt=f32)[::2]),
                     ("state", z(5, K, D)), ("state", z(5, K - 1, D, dt=f32)), ("state", z(5, D)), ("state", None),
                     ("slots", i32([0, 1, 2])), ("slots", i32([0, 1, 2, 3]).long()), ("slots", [0, 1, 2, 3]), ("y", None),
                     ("y", wide[:, 1:D + 1]), ("y", ok["x"]), ("status", z(2, dt=torch.int32)), ("stream", 7)):
        with pytest.raises((A.AttambaError, AttributeError)):
            A.conv_step(**{**ok, key: bad})
    A.conv_step(**{**ok, "x": wide[:, :D], "y": wide[:, D:], "stream": torch.cuda.Stream()})
    seqs = A.Seqs(i32([0, 4]), 4)
    with pytest.raises(A.AttambaError, match="sequence table"):
        A.causal_conv(z(5, D), ok["w"], None, seqs, z(5, D))
    for bad in (i32([0]), i32([[0, 4]]), i32([0, 4]).long(), i32([0, 4]).cpu()):
        with pytest.raises(A.AttambaError, match="cu must"):
            A.Seqs(bad, 4)
    with pytest.raises(A.AttambaError, match="slots must"):
        A.Seqs(i32([0, 4]), 4, slots=i32([0, 1]))
    with pytest.raises(A.AttambaError, match="res must"):
        A.block_norm(z(4, D), z(5, D), z(4, D))
    with pytest.raises(A.AttambaError, match="w_pre must"):
        A.block_norm(z(4, D), z(4, D), z(4, D), z(4, D), w_pre=z(D))
    with pytest.raises(A.AttambaError, match="invalid argument"):
        A.block_norm(z(4, D), z(4, D), z(4, D), eps=-1.0)
    with pytest.raises(TypeError):
        A.block_norm(z(4, D), z(4, D), z(4, D), alpha="x")
    big = scan_inputs(300, D, N, torch.bfloat16, seed=1)
    g = {k: to_gpu(v) for k, v in big.items()}
    with pytest.raises(A.AttambaError, match="workspace"):
        A.selective_scan(*(g[k] for k in ("x", "dt", "bias", "A", "B", "C")), A.Seqs(i32([0, 300]), 300), z(300, D))
    with pytest.raises(A.AttambaError, match="C must"):
        A.scan_step(*(g[k] for k in ("x", "dt", "bias", "A", "B", "x")), z(300, N, D, dt=f32), z(300, D))


def test_other_streams_and_captured_graphs():
    """The prompt and step operators on a side stream, captured into two graphs with a workspace each and replayed
    together, give what the eager calls gave, bit for bit."""
    T, D, N, K = 700, 136, 16, 4
    d = scan_inputs(T, D, N, torch.bfloat16, seed=51)
    g = {k: to_gpu(v) for k, v in d.items()}
    w, bias = torch.randn(D, K, generator=torch.Generator().manual_seed(3)).cuda(), torch.ones(D, device="cuda")
    wn = torch.rand(D, generator=torch.Generator().manual_seed(4)).cuda()
    seqs = A.Seqs(i32(offsets([300, 0, 399])), T, slots=i32([2, 0, 1]), cont=i32([1, 1, 0]))
    start = torch.randn(3, N, D, generator=torch.Generator().manual_seed(5)).cuda()

    def buffers():
        bf = torch.bfloat16
        z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        return dict(st=start.clone(), win=z(3, K - 1, D), c=z(T, D), y=z(T, D), ys=z(3, D), r=z(T, D), h=z(T, D),
                    ws=workspace(T, D, N))

    def block(b):
        A.causal_conv(g["x"], w, bias, seqs, b["c"], state=b["win"])
        A.selective_scan(b["c"], g["dt"], g["bias"], g["A"], g["B"], g["C"], seqs, b["y"], skip=g["skip"], z=g["z"],
                         state=b["st"], workspace=b["ws"])
        A.scan_step(b["c"][:3], g["dt"][:3], g["bias"], g["A"], g["B"][:3], g["C"][:3], b["st"], b["ys"])
        A.block_norm(b["y"], g["x"], b["r"], b["h"], w_post=wn, w_pre=wn)

    eager = buffers()
    block(eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = buffers()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(other)
    torch.cuda.synchronize()
    graphs, sets, streams = [], [buffers(), buffers()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for b in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block(b)
        graphs.append(graph)
    for b in sets:           # capture ran nothing; start from clean state
        b["st"].copy_(start)
        b["win"].zero_()
    torch.cuda.synchronize()
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for b in [other] + sets:
        for k in ("c", "y", "ys", "st", "win", "r", "h"):
            assert torch.equal(b[k], eager[k]), k


# ---------------------------------------------------------------- norm
def norm_bounds(D, y, res, r, h, v, alpha, w_pre, eps, dt, rdt, rel):
    """dr: the sum's rounding and rel of the block's share; h: dr through the norm and the norm's own arithmetic."""
    arith = 48 * U     # a row's sum of squares: at most 72 roundings in a row, half of it after the root; 12 more
    dr = U * (np.abs(r) + (0 if res is None else np.abs(res))) + (rel + arith) * np.abs(alpha * v)
    br = dr + HALF[rdt] * (np.abs(r) + dr) + TINY
    if h is None:
        return br, None
    rms = np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    dn = np.sqrt((dr * dr).sum(axis=1, keepdims=True)) / np.sqrt((r * r).sum(axis=1, keepdims=True) + eps * D)
    bh = np.abs(w_pre) / rms * dr + np.abs(h) * (arith + dn)
    return br, bh + HALF[dt] * (np.abs(h) + bh) + TINY


@pytest.mark.parametrize("D", [8, 72, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768])
@pytest.mark.parametrize("kind", range(8))
def test_block_norm(D, kind):
    M = 5 if D > 600 else 9
    dt, rdt = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32),
               (torch.float32, torch.bfloat16)][kind % 4]
    act = ["silu", "sigmoid", "linear", "silu", "none", "silu", "sigmoid", "none"][kind]
    first, post, pre, has_res, has_scale = kind in (0, 2), kind not in (2, 4), kind != 3, kind != 5, kind in (1, 5)
    g = torch.Generator().manual_seed(D + kind)
    extra = 8 if kind % 2 else 0
    y, res = wide(M, D, dt, g, extra, 2.0), wide(M, D, rdt, g, extra, 3.0) if has_res else None
    gate = wide(M, D, dt, g, extra) if act != "none" else None
    if kind == 0:
        y[1] = 0.0        # a row of zeros: eps alone
    w_post, w_pre = (torch.rand(D, generator=g) + 0.5 if f else None for f in (post, pre))
    scale = torch.randn(D, generator=g) if has_scale else None
    alpha, eps = 0.37, 1e-5
    guard = Guarded()
    r, h = guard((M, D), rdt), guard((M, D), dt) if pre else None
    codes = {"silu": A.ACT_SILU, "sigmoid": A.ACT_SIGMOID, "linear": A.ACT_LINEAR, "none": A.ACT_SILU}
    A.block_norm(to_gpu(y), to_gpu(res), r, h, w_post=to_gpu(w_post), w_pre=to_gpu(w_pre), gate=to_gpu(gate),
                 gate_act=codes[act], gate_first=first, scale=to_gpu(scale), alpha=alpha, eps=eps)
    torch.cuda.synchronize()
    guard.check()
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    kw = dict(w_post=n(w_post), gate=n(gate), act=act if act != "none" else "silu", gate_first=first, scale=n(scale), eps=eps)
    rr, hh = OB.block_norm(n(y), n(res), w_pre=n(w_pre), alpha=np.float32(alpha).astype(np.float64), **kw)
    v, _ = OB.block_norm(n(y), None, **kw)
    # the gate's own error reaches every element of its row through a norm after it: the row's largest
    rel = 0.0 if gate is None else act_bound(kw["act"], n(gate)).max(axis=1, keepdims=True) * (2 if first and post else 1)
    br, bh = norm_bounds(D, n(y), n(res), rr, hh, v, alpha, n(w_pre), eps, dt, rdt, rel)
    assert_within(f64(r), rr, br, "res_out")
    if pre:
        assert_within(f64(h), hh, bh, "h")


def test_block_norm_in_place_and_first_block():
    """res_out on res and h on y give what separate outputs give; without y it is the norm ahead of the first block."""
    M, D = 37, 1032
    g = torch.Generator().manual_seed(1)
    y, res, w = wide(M, D, torch.bfloat16, g).cuda(), wide(M, D, torch.float32, g).cuda(), torch.rand(D, generator=g).cuda()
    r, h = torch.empty_like(res), torch.empty_like(y)
    A.block_norm(y, res, r, h, w_post=w, w_pre=w, alpha=0.5)
    y2, res2 = y.clone(), res.clone()
    A.block_norm(y2, res2, res2, y2, w_post=w, w_pre=w, alpha=0.5)
    assert torch.equal(res2, r) and torch.equal(y2, h)
    h2 = torch.empty_like(h)
    A.block_norm(None, r, None, h2, w_pre=w)
    ref = OB.norm(f64(r), f64(w), 1e-5)
    assert_within(f64(h2), ref, (HALF[torch.bfloat16] + 60 * U) * np.abs(ref) + TINY, "first norm")


def test_block_norm_rows_do_not_mix():
    """Infinities and NaN in one row leave the others as they are."""
    M, D = 11, 520
    g = torch.Generator().manual_seed(2)
    y, res, w = wide(M, D, torch.float32, g).cuda(), wide(M, D, torch.float32, g).cuda(), torch.rand(D, generator=g).cuda()
    out = []
    for bad in (None, float("nan"), float("inf")):
        yy = y.clone()
        if bad is not None:
            yy[4, 100] = bad
        r, h = torch.empty_like(res), torch.empty_like(y)
        A.block_norm(yy, res, r, h, w_post=w, w_pre=w)
        out.append((r, h))
    rows = [i for i in range(M) if i != 4]
    for r, h in out[1:]:
        assert torch.equal(r[rows], out[0][0][rows]) and torch.equal(h[rows], out[0][1][rows])
        assert bool(torch.isnan(h[4]).any())
