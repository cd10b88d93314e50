"""layer.Block on the GPU: a caller's stream, handing a prefill through a block to decoding, the values of its decode steps."""

import math

import numpy as np
import pytest
import torch

from block_cases import HALF, TINY, U, assert_within, offsets, scan_bound
from helpers import f64
from oracle import block as OB
from ssm_compressed_chunked_b200 import attamba as A
from ssm_compressed_chunked_b200 import layer
from ssm_compressed_chunked_b200 import workloads as W
from test_gpu_ssm_block import conv_bound, i32
from test_gpu_ssm_layer import BF, cuda, gemm_check, mixer_weights

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


def norm_of(r, w):
    """The bf16 norm ahead of a mixer, from the operator itself."""
    h = torch.empty(r.shape, dtype=BF, device="cuda")
    A.block_norm(None, r, h=h, w_pre=w)
    return h


def check_join(r, h, y, r0, post, scale, alpha, pre, res):
    """A block's residual sum and next input against the oracle on the mixer's own output."""
    ref, ref_h = OB.block_norm(f64(y), f64(r0), w_post=f64(post), w_pre=f64(pre), scale=f64(scale),
                               alpha=float(np.float32(alpha)))
    v = np.abs(ref - f64(r0))
    # fp32 steps: the norm's sum and root and three products of the block's share, one sum; then the stored rounding
    dr = 60 * U * v + 2 * U * (np.abs(ref) + np.abs(f64(r0)))
    assert_within(f64(r), ref, dr + HALF[res] * (np.abs(ref) + dr) + TINY, "r")
    rms = np.sqrt((ref * ref).mean(axis=1, keepdims=True) + 1e-5)
    rel = np.sqrt((dr * dr).sum(axis=1, keepdims=True) / (ref * ref).sum(axis=1, keepdims=True))
    dh = np.abs(f64(pre)) / rms * dr + np.abs(ref_h) * (60 * U + rel)
    assert_within(f64(h), ref_h, dh + HALF[BF] * (np.abs(ref_h) + dh) + TINY, "h")


@pytest.mark.parametrize("res", [torch.float32, BF])
@pytest.mark.parametrize("N,K,slots", [(16, 4, None), (32, 3, [4, -1, 0, 2, 5])])
def test_block_decode_step_around_the_mixer_has_the_oracles_values(res, N, K, slots):
    """Every stage of a decode step through a block against the oracle, each fed the GPU's own input to it: the norm ahead,
    the mixer's six stages with both states, the join with post-norm, scale and the next block's norm."""
    D, Di, B = 128, 256, 5
    g = torch.Generator().manual_seed(N)
    w = mixer_weights(D, Di, N, K, N)
    mix = layer.SsmMixer(D, Di, N, K, cuda(w), B)
    pre, post, scale, nn = (torch.rand(D, generator=g).cuda() + 0.5 for _ in range(4))
    blk = layer.Block(mix, pre, w_post=post, scale=scale, alpha=0.6)
    win, ssm = mix.new_state(6)
    win.copy_(torch.randn(win.shape, generator=g))
    ssm.copy_(torch.randn(ssm.shape, generator=g))
    r = torch.randn(B, D, generator=g).to(res).cuda()
    live = np.array([s >= 0 for s in (slots or range(B))])
    for _ in range(3):
        r0, win0, ssm0 = r.clone(), win.cpu().clone(), ssm.cpu().clone()
        h0 = norm_of(r0, pre)
        ref = OB.norm(f64(r0), f64(pre), 1e-5)
        assert_within(f64(h0), ref, (HALF[BF] + 60 * U) * np.abs(ref) + TINY, "norm ahead")
        # the mixer called alone on copies of the states gives the y that the block's join read
        y = mix.decode_step((win.clone(), ssm.clone()), h0, slots=i32(slots)).clone()
        r, h = blk.decode_step((win, ssm), r, slots=i32(slots), next_norm=nn)
        assert mix.status.item() == 0
        b = {k: v[:B].cpu()[live] for k, v in mix.buf.items()}
        gemm_check(b["x"], h0.cpu()[live], w["W_in"][:Di], "x")
        gemm_check(b["z"], h0.cpu()[live], w["W_in"][Di:], "z")
        sl = np.asarray(slots if slots else range(B))[live]
        m = int(live.sum())
        args = (f64(b["x"]), f64(w["conv_w"]), f64(w["conv_b"]), offsets([1] * m), f64(win0), sl, np.ones(m, dtype=int))
        lin, _ = OB.causal_conv(*args, act="linear")
        ref, ref_win = OB.causal_conv(*args)
        assert_within(f64(b["u"]), ref, conv_bound(b["x"], w["conv_w"], w["conv_b"], lin, ref, offsets([1] * m), BF, "silu", win0,
                                                   sl, np.ones(m, dtype=int)), "u")
        assert np.array_equal(f64(win), ref_win)
        for name, rows in (("dt", slice(0, Di)), ("B", slice(Di, Di + N)), ("C", slice(Di + N, Di + 2 * N))):
            gemm_check(b[name], b["u"], w["W_x"][rows], name)
        d = dict(x=b["u"], dt=b["dt"], B=b["B"], C=b["C"], z=b["z"], A=w["A"], bias=w["bias"], skip=w["skip"])
        ref, ref_ssm = OB.selective_scan(f64(b["u"]), f64(b["dt"]), f64(w["bias"]), f64(w["A"]), f64(b["B"]), f64(b["C"]),
                                         offsets([1] * m), f64(w["skip"]), f64(b["z"]), f64(ssm0), sl, np.ones(m, dtype=int))
        by, bst = scan_bound(d, offsets([1] * m), BF, ssm0, sl, np.ones(m, dtype=int))
        assert_within(f64(b["s"]), ref, by, "s")
        assert_within(f64(ssm)[sl], ref_ssm[sl], bst[sl], "ssm state")
        gemm_check(y.cpu()[live], b["s"], w["W_O"], "y")
        check_join(r, h, y, r0, post, scale, 0.6, nn, res)


@pytest.mark.parametrize("res", [torch.float32, BF])
def test_block_decode_step_around_the_layer_has_the_oracles_values(res):
    """The layer's own decode step is compared with the oracle elsewhere; here the block's norm ahead of it and the join behind
    it, with the layer called alone on an equal cache."""
    B, H, D = 3, 2, 128
    g = torch.Generator().manual_seed(12)
    lay = attamba_layer(B, 64, H, g)
    pre, post, scale, nn = (torch.rand(D, generator=g).cuda() + 0.5 for _ in range(4))
    blk = layer.Block(lay, pre, w_post=post, scale=scale, alpha=0.6)
    one, two = lay.new_cache(16), lay.new_cache(16)
    r = torch.randn(B, D, generator=g).to(res).cuda()
    for _ in range(10):          # past the first chunk's end
        r0 = r.clone()
        y = lay.decode_step(one, norm_of(r0, pre)).clone()
        r, h = blk.decode_step(two, r, next_norm=nn)
        check_join(r, h, y, r0, post, scale, 0.6, nn, res)
    for k in ("state", "Kb", "Vb", "bpos", "Kr", "Vr", "nb", "pos"):
        assert torch.equal(getattr(one, k), getattr(two, k)), k
    assert lay.status.item() == 0 and int(one.nb.min()) >= 1
