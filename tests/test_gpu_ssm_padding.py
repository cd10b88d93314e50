"""Rows that no sequence owns (behind the last prompt, or of slot -1 in a step): the mixer gives zeros there and a block leaves
the residual stream as it is, whatever its buffers hold."""

import pytest
import torch

from block_cases import offsets
from helpers import Guarded
from ssm_compressed_chunked_b200 import attamba as A
from ssm_compressed_chunked_b200 import layer
from test_gpu_ssm_block import i32
from test_gpu_ssm_layer import BF, cuda, mixer_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("lens,T", [([5, 0, 9], 14), ([5, 0, 9], 15), ([1], 700), ([0], 3), ([2000], 2003), ([3, 4], 7)])
def test_clear_rows_of_a_prompt_batch(dtype, lens, T):
    D, n = 72, sum(lens)
    guard = Guarded()
    y = guard((T, D), dtype)
    y.fill_(3.0)
    A.clear_rows(y, seqs=A.Seqs(i32(offsets(lens)), T))
    torch.cuda.synchronize()
    guard.check()
    assert bool((y[:n] == 3.0).all()) and bool((y[n:] == 0.0).all())


@pytest.mark.parametrize("slots", [[0], [-1], [3, -1, 0, -1, 7], list(range(-1, 1500)), [-1] * 900])
def test_clear_rows_of_a_step(slots):
    D, B = 136, len(slots)
    wide = torch.full((B, 2 * D), 3.0, dtype=BF, device="cuda")
    A.clear_rows(wide[:, D:], slots=i32(slots))
    live = torch.tensor([s >= 0 for s in slots], device="cuda")
    assert bool((wide[:, :D] == 3.0).all()) and bool((wide[live] == 3.0).all()) and bool((wide[~live][:, D:] == 0.0).all())


@pytest.mark.parametrize("cu", [[0, 9, 400], [0, 4, -3], [0, 4, 2 ** 31 - 1], [0, 4, -2 ** 31]])
def test_clear_rows_stays_inside_for_a_malformed_table(cu):
    guard = Guarded()
    y = guard((30, 64), BF)
    A.clear_rows(y, seqs=A.Seqs(i32(cu), 30))
    torch.cuda.synchronize()
    guard.check()


def poisoned_mixer(D, Di, N, K, rows, seed):
    """A mixer whose buffers hold NaN, with a residual block around it."""
    nan = lambda shape, dt: torch.full(shape, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    mix = layer.SsmMixer(D, Di, N, K, cuda(mixer_weights(D, Di, N, K, seed)), rows, alloc=nan)
    g = torch.Generator().manual_seed(seed)
    return mix, layer.Block(mix, torch.rand(D, generator=g).cuda() + 0.5, w_post=torch.rand(D, generator=g).cuda() + 0.5,
                            scale=torch.randn(D, generator=g).cuda(), alpha=0.7)


@pytest.mark.parametrize("res", [torch.float32, BF])
@pytest.mark.parametrize("lens,pad", [([70, 0, 200], 31), ([9], 3), ([0, 0], 20), ([130], 0)])
def test_a_block_leaves_padded_prompt_rows(res, lens, pad):
    D, Di, N, K = 128, 256, 16, 4
    n, T = sum(lens), sum(lens) + pad
    mix, blk = poisoned_mixer(D, Di, N, K, T + 4, seed=T)
    g = torch.Generator().manual_seed(T)
    r0 = torch.randn(T, D, generator=g).to(res).cuda()
    nn = torch.rand(D, generator=g).cuda() + 0.5
    r, h = blk.forward(r0.clone(), A.Seqs(i32(offsets(lens)), T), next_norm=nn)
    assert torch.equal(r[n:], r0[n:])
    assert bool(torch.isfinite(r.float()).all()) and bool(torch.isfinite(h.float()).all())
    assert n == 0 or not torch.equal(r[:n], r0[:n])
    want = torch.empty(T, D, dtype=BF, device="cuda")
    A.block_norm(None, r0, h=want, w_pre=nn)
    assert torch.equal(h[n:], want[n:])          # the next block's input there is the norm of the row as it was
    assert bool((mix.forward(h, A.Seqs(i32(offsets(lens)), T))[n:] == 0.0).all()) and mix.status.item() == 0


@pytest.mark.parametrize("res", [torch.float32, BF])
def test_a_block_leaves_padded_decode_rows(res):
    """Also replayed from a captured graph that works on one residual buffer, with buffers that hold NaN."""
    D, Di, N, K, B = 128, 256, 32, 3, 6
    mix, blk = poisoned_mixer(D, Di, N, K, 16, seed=4)
    slots, state = i32([2, -1, 0, -1, 3, 1]), mix.new_state(4)
    pad, live = [1, 3], [0, 2, 4, 5]
    r0 = torch.randn(B, D, generator=torch.Generator().manual_seed(6)).to(res).cuda()
    r = r0.clone()
    blk.decode_step(state, r, slots=slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.decode_step(state, r, slots=slots)
    for buf in mix.buf.values():
        buf.fill_(float("nan"))
    for _ in range(3):
        before = r.clone()
        graph.replay()
        assert torch.equal(r[pad], r0[pad]) and bool(torch.isfinite(r.float()).all()) and not torch.equal(r[live], before[live])
    assert mix.status.item() == 0
