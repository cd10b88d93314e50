"""The single-token steps where a block walks several batch rows, and the prompt scan's join over many tiles: what batches of
hundreds of rows and long narrow prompts run, against the float64 oracle."""

import numpy as np
import pytest
import torch

from block_cases import DT, assert_within, offsets, scan_bound, scan_inputs, to_gpu, wide
from helpers import f64
from oracle import block as OB
from ssm_compressed_chunked_b200 import attamba as A
from test_gpu_ssm_block import conv_bound, i32, new_status, run_scan
from test_gpu_ssm_wide import channels_of

pytestmark = pytest.mark.gpu


def colliding_slots(B, n_slots, seed):
    """Different slots, half of them equal mod 256 (the slot search's table has 256 entries), with rows that only fill the
    batch up between them."""
    rng = np.random.default_rng(seed)
    same = np.arange(3, n_slots, 256)[:B // 2]
    rest = rng.permutation(np.setdiff1d(np.arange(n_slots), same))[:B - len(same)]
    slots = rng.permutation(np.concatenate([same, rest])).astype(np.int64)
    slots[[1, B // 2, B // 2 + 1, B - 7]] = -1
    return slots


# rows a block walks (148 SMs, 6 or 3 blocks each, 128 channels a block): 5, 5, 40, 22, 2
STEP = [("bf16", 256, 2048, 16), ("f32", 256, 2048, 16), ("bf16", 512, 4096, 32), ("f32", 130, 8200, 32), ("bf16", 1500, 72, 16)]


def step_case(dtype, B, D, N, slots, n_slots):
    """One scan_step on the GPU with poisoned outputs -> (inputs, state before, y, state after, status)."""
    d = scan_inputs(B, D, N, DT[dtype], seed=B + D)
    g = torch.Generator(device="cuda").manual_seed(B)
    state = torch.randn(n_slots, N, D, generator=g, device="cuda")
    st, status = state.clone(), new_status()
    y = torch.full((B, D), float("nan"), dtype=DT[dtype], device="cuda")
    A.scan_step(*(to_gpu(d[k]) for k in ("x", "dt", "bias", "A", "B", "C")), st, y, skip=to_gpu(d["skip"]), z=to_gpu(d["z"]),
                slots=i32(slots), status=status)
    torch.cuda.synchronize()
    return d, state, y, st, status.item()


def check_step(dtype, D, d, state, y, st, slots):
    """y and states of the rows with a slot against the oracle on sampled channels; all else untouched."""
    slots = np.asarray(slots)
    live = slots >= 0
    used = slots[live]
    pick = sorted({0, 1, 4, 7, 31, 32, 63, 71, D // 2 - 1, D // 2, D - 2, D - 1} & set(range(D)))
    part = channels_of(d, pick)
    n = {k: f64(v) for k, v in part.items()}
    rows = {k: (v[live] if k in ("x", "dt", "B", "C", "z") else v) for k, v in part.items()}
    m = int(live.sum())
    cu, cont = offsets([1] * m), np.ones(m, dtype=int)
    init = state[torch.from_numpy(used).cuda()][:, :, pick].cpu()
    ref, ref_st = OB.selective_scan(*(n[k][live] for k in ("x", "dt")), n["bias"], n["A"], n["B"][live], n["C"][live], cu,
                                    n["skip"], n["z"][live], f64(init), None, cont)
    by, bst = scan_bound(rows, cu, DT[dtype], init, None, cont)
    mask = torch.from_numpy(live).cuda()
    assert_within(f64(y[mask][:, pick]), ref, by, "y")
    got = st[torch.from_numpy(used).cuda()]
    assert_within(f64(got[:, :, pick]), ref_st, bst, "state")
    assert bool(torch.isfinite(y[mask].float()).all()) and bool(torch.isnan(y[~mask]).all())
    rest = torch.ones(state.shape[0], dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(used).cuda()] = False
    assert torch.equal(st[rest], state[rest]), "rows of no sequence stay as they were"


@pytest.mark.parametrize("dtype,B,D,N", STEP)
def test_scan_step_of_many_rows(dtype, B, D, N):
    n_slots = min(2048, max(B + 9, (1 << 28) // (N * D)))
    slots = colliding_slots(B, n_slots, B)
    d, state, y, st, status = step_case(dtype, B, D, N, slots, n_slots)
    assert status == 0
    check_step(dtype, D, d, state, y, st, slots)


# (row, its earlier twin): rows r and r + k * 52 of the first case are one block's, r and r + k * 13 of the third's, where
# row 458 is the 36th of its block
@pytest.mark.parametrize("case,twins", [(0, [(62, 10), (218, 10), (200, 11), (255, 254)]), (2, [(458, 3), (16, 3), (511, 510), (400, 7)]),
                                        (4, [(1499, 0), (800, 2), (801, 2)])])
def test_scan_step_repeated_slots_among_many_rows(case, twins):
    dtype, B, D, N = STEP[case]
    n_slots = min(2048, max(B + 9, (1 << 28) // (N * D)))
    slots = colliding_slots(B, n_slots, B + 1)
    free = np.setdiff1d(np.arange(n_slots), slots)
    for k, (late, early) in enumerate(twins):
        if slots[early] < 0:
            slots[early] = free[k]
        slots[late] = slots[early]
    wrong = 30
    slots[wrong] = n_slots + 256
    d, state, y, st, status = step_case(dtype, B, D, N, slots, n_slots)
    assert status == A.DEV_BAD_SEQS
    kept = slots.copy()
    kept[[late for late, _ in twins] + [wrong]] = -1          # skipped: neither their y nor a state row is written
    check_step(dtype, D, d, state, y, st, kept)


@pytest.mark.parametrize("dtype,B,D,K", [("bf16", 512, 264, 4), ("f32", 333, 136, 2)])
def test_conv_step_of_many_rows_with_repeated_slots(dtype, B, D, K):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(B)
    n_slots = 4096
    slots = colliding_slots(B, n_slots, B)
    for late, early in ((B - 1, B - 2), (200, 5), (7, 6), (300, 5)):
        if slots[early] < 0:
            slots[early] = 4095
        slots[late] = slots[early]
    kept = slots.copy()
    kept[[B - 1, 200, 7, 300]] = -1
    x, w = wide(B, D, dt, g), torch.randn(D, K, generator=g)
    state = torch.randn(n_slots, K - 1, D, generator=g).to(dt)
    st, status = state.cuda(), new_status()
    y = torch.full((B, D), float("nan"), dtype=dt, device="cuda")
    A.conv_step(x.cuda(), w.cuda(), None, st, y, slots=i32(slots), status=status)
    torch.cuda.synchronize()
    assert status.item() == A.DEV_BAD_SEQS
    args = (f64(x), f64(w), None, offsets([1] * B), f64(state), kept, np.ones(B, dtype=int))
    pre, _ = OB.causal_conv(*args, act="linear")
    ref, ref_st = OB.causal_conv(*args)
    live = kept >= 0
    b = conv_bound(x, w, None, pre, ref, offsets([1] * B), dt, "silu", state, kept, np.ones(B, dtype=int))
    assert_within(f64(y)[live], ref[live], b[live], "y")
    assert bool(torch.isnan(y[torch.from_numpy(~live).cuda()]).all()) and np.array_equal(f64(st), ref_st)


# ---------------------------------------------------------------- the join of many tiles
def slow_decays(d):
    """Steps so small that a prompt's first tokens still count at its end."""
    d["bias"] = torch.full_like(d["bias"], -9.0)
    d["dt"] = d["dt"] * 0.1
    d["A"] = d["A"] / 16
    return d


# 8192 x 64: N 16 in 357 tiles of 23 tokens, N 32 in 512 of 16 (148 SMs, five blocks each, two of them a tile; four, one a
# tile). A join walks 128 tiles (2944 or 2048 tokens) at a time: sequences across all of them, and with ends at, just ahead
# of and just behind the 128th and the 256th
@pytest.mark.parametrize("N,lens", [(16, [8192]), (16, [2944, 5248]), (16, [2943, 2, 2943, 2304]), (16, [2945, 0, 5247]),
                                    (16, [1472, 4416, 2304]), (32, [8192]), (32, [2048, 6144]), (32, [2047, 2049, 4096])])
def test_scan_across_more_tiles_than_a_join_walks_at_once(N, lens):
    T, D = sum(lens), 64
    d = slow_decays(scan_inputs(T, D, N, torch.float32, seed=len(lens) + N))
    cu, S = offsets(lens), len(lens)
    state = torch.randn(S, N, D, generator=torch.Generator().manual_seed(S)) * 30     # large: it is felt to the end
    cont = np.ones(S, dtype=int)
    y, st, status = run_scan(d, cu, T, torch.float32, state, None, cont)
    assert status == 0
    pick = [0, 1, 17, 31, 32, 33, 62, 63]
    part = channels_of(d, pick)
    n = {k: f64(v) for k, v in part.items()}
    ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], cu, n["skip"], n["z"],
                                    f64(state[:, :, pick]), None, cont)
    by, bst = scan_bound(part, cu, torch.float32, state[:, :, pick], None, cont)
    assert_within(f64(y[:, pick]), ref, by, "y")
    assert_within(f64(st[:, :, pick]), ref_st, bst, "state")
    # the inputs can tell (oracle alone): with the carried state lost half of the last rows would be off by more than twice
    # their bound, so that no error within the bound hides it
    last = int(cu[-2])
    if T - last > 5900:
        lost, _ = OB.selective_scan(n["x"][last:], n["dt"][last:], n["bias"], n["A"], n["B"][last:], n["C"][last:], [0, T - last],
                                    n["skip"], n["z"][last:])
        off = np.abs(lost - ref[last:]) / by[last:]
        assert np.median(off[-500:]) > 2


# ---------------------------------------------------------------- the documented limits
def gpu_inputs(T, D, N, seed):
    """scan_inputs' distributions in bf16, made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=n(T, D), dt=n(T, D), B=n(T, N), C=n(T, N), z=n(T, D), A=-torch.exp(u(D, N) * np.log(16.0)), skip=u(D) - 0.5,
                bias=torch.log(torch.expm1(torch.exp(u(D) * np.log(100.0) + np.log(1e-3)))))


@pytest.mark.parametrize("T,lens", [(3, [2, 1]), (130, [100, 0, 29])])
def test_the_widest_rows(T, lens):
    """2^20 channels, the most that a call takes: prompts in a single tile of one or many windows, and steps."""
    D, N, K, S = 1 << 20, 16, 4, len(lens)
    bf = torch.bfloat16
    d = gpu_inputs(T, D, N, T)
    cu, cont = offsets(lens), [1] * S
    g = torch.Generator(device="cuda").manual_seed(1)
    state = torch.randn(S, N, D, generator=g, device="cuda")
    win = torch.randn(S, K - 1, D, generator=g, device="cuda").to(bf)
    w = torch.randn(D, K, generator=g, device="cuda")
    seqs, status = A.Seqs(i32(cu), T, cont=i32(cont)), new_status()
    ws = A.selective_scan_workspace_size(T, D, N)
    y, cy = torch.full((T, D), float("nan"), dtype=bf, device="cuda"), torch.full((T, D), float("nan"), dtype=bf, device="cuda")
    st, wn = state.clone(), win.clone()
    A.selective_scan(d["x"], d["dt"], d["bias"], d["A"], d["B"], d["C"], seqs, y, skip=d["skip"], z=d["z"], state=st,
                     workspace=torch.empty(ws, dtype=torch.uint8, device="cuda") if ws else None, status=status)
    A.causal_conv(d["x"], w, None, seqs, cy, state=wn, status=status)
    ys, cs = torch.full((S, D), float("nan"), dtype=bf, device="cuda"), torch.full((S, D), float("nan"), dtype=bf, device="cuda")
    st1, wn1 = state.clone(), win.clone()
    A.scan_step(d["x"][:S], d["dt"][:S], d["bias"], d["A"], d["B"][:S], d["C"][:S], st1, ys, skip=d["skip"], z=d["z"][:S],
                status=status)
    A.conv_step(d["x"][:S], w, None, wn1, cs, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    pick = [0, 1, 255, 256, 4095, 4096, D // 2 - 1, D // 2, D - 129, D - 128, D - 2, D - 1]
    part = {k: v.cpu() for k, v in channels_of(d, pick).items()}
    init, iw, pw = state[:, :, pick].cpu(), win[:, :, pick].cpu(), w[pick].cpu()
    m = sum(lens)
    for rows, tab, got_y, got_st, got_c, got_w in ((T, cu, y, st, cy, wn), (S, offsets([1] * S), ys, st1, cs, wn1)):
        p = {k: (v[:rows] if k in ("x", "dt", "B", "C", "z") else v) for k, v in part.items()}
        n = {k: f64(v) for k, v in p.items()}
        live = min(m, rows)
        ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], tab, n["skip"], n["z"], f64(init),
                                        None, cont)
        by, bst = scan_bound(p, tab, bf, init, None, cont)
        assert_within(f64(got_y[:live, pick]), ref[:live], by[:live], "scan y")
        assert_within(f64(got_st[:, :, pick]), ref_st, bst, "scan state")
        pre, _ = OB.causal_conv(n["x"], f64(pw), None, tab, f64(iw), None, cont, act="linear")
        ref, ref_w = OB.causal_conv(n["x"], f64(pw), None, tab, f64(iw), None, cont)
        b = conv_bound(p["x"], pw, None, pre, ref, tab, bf, "silu", iw, None, cont)
        assert_within(f64(got_c[:live, pick]), ref[:live], b[:live], "conv y")
        assert np.array_equal(f64(got_w[:, :, pick]), ref_w)
    assert bool(torch.isnan(y[m:]).all()) and bool(torch.isnan(cy[m:]).all())
    assert not bool(torch.isnan(y[:m]).any()) and not bool(torch.isnan(cy[:m]).any())


def test_the_most_sequences():
    """2^20 sequences of no, one and two tokens without a slot map, half of them continuing; compared on samples from both
    ends and between."""
    S, D, N, K = 1 << 20, 8, 16, 4
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 3, S)
    lens[-40:] = 0
    cu = offsets(lens)
    T = int(cu[-1]) + 5
    cont = rng.integers(0, 2, S)
    d = gpu_inputs(T, D, N, 9)
    g = torch.Generator(device="cuda").manual_seed(2)
    state = torch.randn(S, N, D, generator=g, device="cuda")
    win = torch.randn(S, K - 1, D, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(D, K, generator=g, device="cuda")
    seqs, status = A.Seqs(i32(cu), T, cont=i32(cont)), new_status()
    y, cy = (torch.full((T, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st, wn = state.clone(), win.clone()
    ws = torch.empty(A.selective_scan_workspace_size(T, D, N), dtype=torch.uint8, device="cuda")
    A.selective_scan(d["x"], d["dt"], d["bias"], d["A"], d["B"], d["C"], seqs, y, skip=d["skip"], z=d["z"], state=st,
                     workspace=ws, status=status)
    A.causal_conv(d["x"], w, None, seqs, cy, state=wn, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and bool(torch.isnan(y[T - 5:]).all()) and not bool(torch.isnan(y[:T - 5]).any())
    for a in (0, S // 3, S // 2 + 17, S - 300):
        b = a + 300
        t0, t1 = int(cu[a]), int(cu[b])
        sub, c = (cu[a:b + 1] - t0).astype(np.int32), cont[a:b]
        p = {k: (v[t0:t1] if k in ("x", "dt", "B", "C", "z") else v).cpu() for k, v in d.items()}
        n = {k: f64(v) for k, v in p.items()}
        init, iw = state[a:b].cpu(), win[a:b].cpu()
        ref, ref_st = OB.selective_scan(n["x"], n["dt"], n["bias"], n["A"], n["B"], n["C"], sub, n["skip"], n["z"], f64(init),
                                        None, c)
        by, bst = scan_bound(p, sub, torch.bfloat16, init, None, c)
        assert_within(f64(y[t0:t1]), ref, by, "scan y")
        assert_within(f64(st[a:b]), ref_st, bst, "scan state")
        pre, _ = OB.causal_conv(n["x"], f64(w), None, sub, f64(iw), None, c, act="linear")
        ref, ref_w = OB.causal_conv(n["x"], f64(w), None, sub, f64(iw), None, c)
        assert_within(f64(cy[t0:t1]), ref, conv_bound(p["x"], w.cpu(), None, pre, ref, sub, torch.bfloat16, "silu", iw, None, c),
                      "conv y")
        assert np.array_equal(f64(wn[a:b]), ref_w)
