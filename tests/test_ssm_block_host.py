"""Refusals of the SSM block's operators, on the host: the C ABI rejects bad arguments before any launch and the
binding rejects CPU tensors (no GPU needed)."""

import ctypes

import pytest
import torch

from ssm_compressed_chunked_b200 import attamba as A

FAKE = 1 << 20            # an aligned address that is never read
FAR = 1 << 40             # outputs: far from the inputs, so that no range check joins them
INV, UNS = A.ERR_INVALID_ARG, A.ERR_UNSUPPORTED


def _seqs(cu=FAKE, slots=None, cont=None, T=16, S=2):
    return ctypes.byref(A.SeqsT(cu, slots, cont, T, S))


def _conv(dtype=A.BF16, x=FAKE, ldx=64, w=FAKE, bias=None, D=64, K=4, act=A.ACT_SILU, seqs=None, state=None, n=0, y=FAR,
          ldy=64):
    return A.load().attamba_causal_conv(dtype, x, ldx, w, bias, D, K, act, seqs or _seqs(), state, n, y, ldy, None, None)


def _conv_step(dtype=A.BF16, x=FAKE, ldx=64, w=FAKE, D=64, K=4, act=A.ACT_SILU, B=4, slots=None, state=2 * FAR, n=4, y=FAR,
               ldy=64):
    return A.load().attamba_conv_step(dtype, x, ldx, w, None, D, K, act, B, slots, state, n, y, ldy, None, None)


def _scan(dtype=A.BF16, x=FAKE, ldx=64, dt=FAKE, Aw=FAKE, B=FAKE, ldb=16, z=None, ldz=64, D=64, N=16, seqs=None,
          state=None, n=0, y=FAR, ldy=64, ws=None, size=0):
    return A.load().attamba_selective_scan(dtype, x, ldx, dt, 64, None, Aw, B, ldb, FAKE, 16, None, z, ldz, D, N,
                                           seqs or _seqs(), state, n, y, ldy, ws, size, None, None)


def _scan_step(dtype=A.BF16, x=FAKE, D=64, N=16, rows=4, state=2 * FAR, n=4, y=FAR):
    return A.load().attamba_scan_step(dtype, x, D, FAKE, D, None, FAKE, FAKE, N, FAKE, N, None, None, 0, D, N, rows, None,
                                      state, n, y, D, None, None)


def _norm(dtype=A.BF16, rdtype=A.BF16, y=FAKE, ldy=64, gate=None, ldg=64, act=A.ACT_SILU, w_post=None, res=3 * FAR,
          ldr=64, scale=None, w_pre=FAKE, eps=1e-5, M=4, D=64, out=FAR, ldo=64, h=2 * FAR, ldh=64):
    return A.load().attamba_block_norm(dtype, rdtype, y, ldy, gate, ldg, act, 0, w_post, res, ldr, scale, 1.0, w_pre,
                                       eps, M, D, out, ldo, h, ldh, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), UNS), (dict(K=1), UNS), (dict(K=5), UNS), (dict(D=60), INV), (dict(D=0), INV),
    (dict(act=A.ACT_SIGMOID), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV),
    (dict(x=FAKE + 2), INV), (dict(w=FAKE + 4), INV), (dict(bias=FAKE + 4), INV), (dict(y=FAR + 8), INV),
    (dict(ldx=56), INV), (dict(ldx=68), INV), (dict(ldy=60), INV), (dict(ldx=1 << 31), INV),
    (dict(seqs=_seqs(T=0)), INV), (dict(seqs=_seqs(S=0)), INV), (dict(seqs=_seqs(cu=None)), INV),
    (dict(seqs=_seqs(T=1 << 31)), INV), (dict(state=2 * FAR, n=0), INV), (dict(state=2 * FAR + 2, n=4), INV),
    (dict(y=FAKE), INV), (dict(y=FAKE + 64 * 2 * 15), INV),                     # y on x, y on x's last row
    (dict(x=FAKE, ldx=128, y=FAKE + 112, ldy=128), INV),                        # column windows that cut each other
    (dict(state=FAR, n=1), INV), (dict(state=FAKE, n=1), INV)])                 # state on y, on x
def test_causal_conv_refuses(kw, code):
    assert _conv(**kw) == code


@pytest.mark.parametrize("kw,code", [(dict(state=None), INV), (dict(B=0), INV), (dict(n=0), INV), (dict(K=5), UNS),
                                     (dict(D=4), INV), (dict(y=2 * FAR), INV), (dict(dtype=3), UNS)])
def test_conv_step_refuses(kw, code):
    assert _conv_step(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNS), (dict(N=24), UNS), (dict(N=64), UNS), (dict(D=12), INV), (dict(x=None), INV), (dict(dt=None), INV),
    (dict(Aw=None), INV), (dict(B=None), INV), (dict(y=None), INV), (dict(Aw=FAKE + 4), INV), (dict(ldb=12), INV),
    (dict(ldb=20), INV), (dict(z=FAKE + 4), INV), (dict(z=FAKE, ldz=8), INV), (dict(y=FAKE), INV),
    (dict(z=FAR), INV), (dict(state=2 * FAR, n=0), INV), (dict(state=FAR, n=2), INV),
    (dict(seqs=_seqs(T=4096), ws=None), INV),                                   # needs a workspace
    (dict(seqs=_seqs(T=4096), ws=3 * FAR, size=1024), INV), (dict(seqs=_seqs(T=4096), ws=3 * FAR + 4, size=1 << 30), INV)])
def test_selective_scan_refuses(kw, code):
    assert _scan(**kw) == code


def test_every_refusal_says_why():
    """The thread's error text is the reason of the refusal at hand, not one left from before."""
    err = lambda: A.load().attamba_last_error().decode()  # noqa: E731
    for call, kw, why in ((_conv, dict(K=5), "K is"), (_conv, dict(y=FAKE), "y overlaps x"), (_conv, dict(D=60), "D is"),
                          (_conv, dict(seqs=_seqs(T=0)), "sequence table"), (_conv_step, dict(state=None), "a state"),
                          (_scan, dict(N=24), "N is"), (_scan, dict(dt=None), "required"), (_scan, dict(Aw=FAKE + 4), "aligned"),
                          (_scan, dict(ldb=12), "row stride"), (_scan_step, dict(n=0), "slot"), (_norm, dict(eps=-1.0), "eps"),
                          (_norm, dict(h=None), "go together"), (_norm, dict(D=32776), "32768"), (_norm, dict(act=3), "act is")):
        assert call(**kw) in (INV, UNS)
        assert why in err() and err().startswith("attamba_"), (kw, err())


def test_more_sequences_than_a_call_takes_are_refused():
    many, slots = (1 << 20) + 1, FAKE
    assert _conv(seqs=_seqs(S=many)) == UNS and _scan(seqs=_seqs(S=many)) == UNS
    assert _conv(seqs=_seqs(S=8193, slots=slots)) == UNS and _scan(seqs=_seqs(S=8193, slots=slots)) == UNS
    assert b"at most 8192 with slots" in A.load().attamba_last_error()
    assert _conv_step(B=many) == UNS and _conv_step(B=8193, slots=slots) == UNS
    assert _scan_step(rows=many) == UNS


def test_selective_scan_says_how_much_workspace_it_needs():
    assert _scan(seqs=_seqs(T=4096)) == INV
    assert b"bytes of workspace" in A.load().attamba_last_error()
    size = A.selective_scan_workspace_size
    assert size(4096, 64, 16) > 0 and size(4096, 64, 32) > size(4096, 64, 16)
    for D, N in ((64, 16), (264, 16), (1024, 16), (1024, 32), (8192, 32)):
        sizes = [size(T, D, N) for T in [*range(1, 400), *range(400, 70000, 97), 1 << 20, 1 << 30]]
        assert sizes == sorted(sizes) and sizes[0] == 0
    assert size(0, 64, 16) == 0 and size(4096, 60, 16) == 0 and size(4096, 64, 8) == 0 and size(1 << 31, 64, 16) == 0


@pytest.mark.parametrize("kw,code", [(dict(state=None), INV), (dict(rows=0), INV), (dict(n=0), INV), (dict(N=8), UNS),
                                     (dict(y=2 * FAR), INV), (dict(y=FAKE), INV), (dict(D=20), INV)])
def test_scan_step_refuses(kw, code):
    assert _scan_step(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), UNS), (dict(rdtype=5), UNS), (dict(D=32776), UNS), (dict(D=20), INV), (dict(M=0), INV),
    (dict(M=1 << 31), INV), (dict(y=None, res=None), INV), (dict(out=None, h=None, w_pre=None), INV), (dict(w_pre=None), INV),
    (dict(h=None), INV), (dict(y=None, gate=FAKE), INV), (dict(y=None, w_post=FAKE), INV), (dict(y=None, scale=FAKE), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(act=3), INV), (dict(w_pre=FAKE + 4), INV), (dict(ldy=63), INV),
    (dict(gate=FAKE, ldg=60), INV), (dict(out=FAKE), INV), (dict(out=3 * FAR, ldo=128), INV), (dict(h=FAKE, ldh=128), INV),
    (dict(h=FAR), INV), (dict(gate=FAR), INV), (dict(rdtype=A.F32, out=3 * FAR + 128), INV)])
def test_block_norm_refuses(kw, code):
    assert _norm(**kw) == code


def test_the_binding_refuses_cpu_tensors_and_other_objects():
    x = torch.zeros(4, 64)
    w, st = torch.zeros(64, 4), torch.zeros(4, 3, 64)
    with pytest.raises(A.AttambaError, match="CUDA"):
        A.conv_step(x, w, None, st, torch.zeros(4, 64))
    with pytest.raises(A.AttambaError, match="CUDA"):
        A.Seqs(torch.tensor([0, 4], dtype=torch.int32), 4)
    with pytest.raises(A.AttambaError, match="CUDA"):
        A.scan_step(x, x, None, torch.zeros(64, 16), torch.zeros(4, 16), torch.zeros(4, 16), torch.zeros(4, 16, 64), x)
    with pytest.raises(A.AttambaError, match="CUDA"):
        A.block_norm(x, x, x)
    with pytest.raises(A.AttambaError, match="y or res"):
        A.block_norm(None, None, x)
    with pytest.raises(A.AttambaError, match="x must be a tensor"):
        A.conv_step(None, w, None, st, x)
    with pytest.raises(A.AttambaError, match="w must be a tensor|CUDA"):
        A.conv_step(x, [1, 2], None, st, x)


def test_the_binding_shares_the_process_cxx_runtime():
    """The marshalling module needs the C++ runtime as a shared library, like torch: a copy of its own linked in would
    be a second one in the process, whose exceptions and locales are not the first's."""
    import subprocess
    from ssm_compressed_chunked_b200 import build
    out = subprocess.run(["readelf", "-d", build.BINDING], capture_output=True, text=True, check=True).stdout
    assert "libstdc++.so" in out and "libtorch_python.so" in out
