"""layer.Block on the GPU beyond the plain call: a caller's stream, handing a prefill through a block to decoding."""

import math

import pytest
import torch

from block_cases import offsets
from helpers import f64
from ssm_compressed_chunked_b200 import attamba as A
from ssm_compressed_chunked_b200 import layer
from ssm_compressed_chunked_b200 import workloads as W
from test_gpu_ssm_block import i32
from test_gpu_ssm_layer import BF, cuda, mixer_weights

pytestmark = pytest.mark.gpu


def attamba_layer(B, n, H, g):
    """A Layer of the inference-mask workload's kind with random weights."""
    D, N = 64 * H, 16
    cfg = W.shrink(W.BF16_TEST_P8_L64, B=B, n=n, D=D, H=H)
    inp = W.make_layer(cfg)
    shapes = {"W_Q": (D, D), "W_dtK": (D, D), "W_dtV": (D, D), "W_BK": (N, D), "W_CK": (N, D), "W_BV": (N, D),
              "W_CV": (N, D), "W_O": (D, D)}
    w = {k: (torch.randn(*s, generator=g) / math.sqrt(D)).to(BF).cuda() for k, s in shapes.items()}
    w.update({k: inp[k].cuda() for k in ("bias_k", "bias_v", "A_k", "A_v")})
    return layer.Layer(B, n, D, H, 64, N, w, cfg.P, cfg.offset, cfg.L, A.MASK_TEST, inp["scale"])


def test_block_on_a_side_stream():
    """forward and decode_step queued on a busy side stream while the current stream allocates and fills tensors of the
    block's input's size: the same rows and states as the calls on the current stream."""
    D, Di, N, K, B = 128, 256, 16, 4, 4
    lens = [90, 0, 41, 130]
    T = sum(lens)
    g = torch.Generator().manual_seed(1)
    w, norm = cuda(mixer_weights(D, Di, N, K, 3)), torch.rand(D, generator=g).cuda() + 0.5
    seqs = A.Seqs(i32(offsets(lens)), T)
    r0, t0 = torch.randn(T, D, generator=g).cuda(), torch.randn(B, D, generator=g).cuda()
    results = []
    for side in (None, torch.cuda.Stream()):
        mix = layer.SsmMixer(D, Di, N, K, w, T)
        blk, state = layer.Block(mix, norm), mix.new_state(B)
        r, t = r0.clone(), t0.clone()
        torch.cuda.synchronize()
        if side is not None:
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)       # a bounded spin of about 10 ms
        for _ in range(3):
            blk.forward(r, seqs, state=state, stream=side)
            blk.decode_step(state, t, stream=side)
            for n in (T, B):
                for _ in range(8):
                    torch.full((n, D), float("nan"), dtype=BF, device="cuda")
        torch.cuda.synchronize()
        assert mix.status.item() == 0
        results.append((r, t, *state))
    assert bool(torch.isfinite(results[0][0]).all())
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_prefill_through_a_block_hands_over_to_decoding():
    """A block around the Attamba layer keeps the layer's input: a cache made from it is the one made from the layer
    called alone, also after another sequence's decode step through the block, and decoding goes on from it."""
    B, n, H = 2, 96, 2
    g = torch.Generator().manual_seed(8)
    lay = attamba_layer(B, n, H, g)
    D = 64 * H
    norm = torch.rand(D, generator=g).cuda() + 0.5
    blk = layer.Block(lay, norm)
    r0, t0 = torch.randn(B * n, D, generator=g).cuda(), torch.randn(B, D, generator=g).cuda()
    x = torch.empty(B * n, D, dtype=BF, device="cuda")
    A.block_norm(None, r0, h=x, w_pre=norm)
    lay.forward(x)
    want = lay.new_cache(32)
    lay.cache_from_prefill(want, x)
    blk.forward(r0.clone())
    assert torch.equal(blk.h, x)
    blk.decode_step(lay.new_cache(32), t0.clone())
    got = lay.new_cache(32)
    lay.cache_from_prefill(got, blk.h)
    for k in ("state", "Kb", "Vb", "bpos", "Kr", "Vr", "nb", "pos"):
        assert torch.equal(getattr(got, k), getattr(want, k)), k
    a, _ = blk.decode_step(got, t0.clone())
    b, _ = blk.decode_step(want, t0.clone())
    assert torch.equal(a, b) and lay.status.item() == 0 and bool(f64(a).any())
