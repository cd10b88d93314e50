"""layer.SsmMixer and layer.Block on the host (no GPU): which buffers they use and keep, with the library's calls replaced by
recorders."""

import pytest
import torch

from ssm_compressed_chunked_b200 import attamba as A
from ssm_compressed_chunked_b200 import layer

BF = torch.bfloat16


class Mixer:
    """A mixer that records what it is handed and returns its own buffer."""

    def __init__(self, rows, D):
        self.y, self.seen = torch.zeros(rows, D, dtype=BF), []

    def forward(self, h, stream=None):
        self.seen.append(h)
        return self.y[:h.shape[0]]

    def decode_step(self, cache, h, stream=None):
        self.seen.append(h)
        return self.y[:h.shape[0]]


@pytest.fixture
def norms(monkeypatch):
    """attamba.block_norm as a recorder of its h argument."""
    calls = []
    monkeypatch.setattr(A, "block_norm", lambda y, res, res_out=None, h=None, **kw: calls.append(h))
    return calls


def count_allocations(monkeypatch):
    made = []
    for name in ("empty", "zeros", "empty_like"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, _f=real, **kw: made.append(1) or _f(*a, **kw))
    return made


def test_block_keeps_its_input_buffer(norms, monkeypatch):
    """The first call makes the block's input buffer; later ones of that many rows or fewer allocate nothing and use the
    same memory, so that nothing goes back to an allocator while a stream still reads it."""
    D = 64
    mix = Mixer(32, D)
    blk = layer.Block(mix, torch.ones(D))
    r = torch.zeros(20, D)
    blk.forward(r)
    blk.decode_step(None, r[:5])
    made = count_allocations(monkeypatch)
    blk.forward(r)
    blk.forward(r[:7])
    blk.decode_step(None, r[:5])
    blk.decode_step(None, r[:3])
    assert not made
    at = [h.data_ptr() for h in mix.seen]
    assert at[0] == at[2] == at[3] and at[1] == at[4] == at[5] and at[0] != at[1]
    assert [h.shape[0] for h in mix.seen] == [20, 5, 20, 7, 5, 3] and all(h.dtype == BF for h in mix.seen)


def test_block_keeps_every_buffer_it_has_handed_out(norms):
    """A captured graph holds the address of the buffer that its capture saw: a larger call makes another one and frees
    none."""
    D = 64
    mix = Mixer(4096, D)
    blk = layer.Block(mix, torch.ones(D))
    sizes = [1, 3, 2, 100, 5, 4096, 100]
    taken = []
    for n in sizes:
        blk.decode_step(None, torch.zeros(n, D))
        h = mix.seen[-1]
        taken.append((h.data_ptr(), h.data_ptr() + h.numel() * h.element_size()))
        mix.seen.clear()
        other = torch.full((n, D), 7.0, dtype=BF)          # fresh memory of the same size lies in none of them
        a = other.data_ptr()
        assert all(a + other.numel() * 2 <= lo or a >= hi for lo, hi in taken)
    assert taken[5][0] == taken[6][0]


def test_block_of_a_mixer_with_a_capacity_makes_one_buffer(norms):
    D = 64
    mix = Mixer(128, D)
    mix.max_tokens = 100
    blk = layer.Block(mix, torch.ones(D))
    at = set()
    for n in (100, 1, 70, 100):
        blk.forward(torch.zeros(n, D))
        at.add(mix.seen[-1].data_ptr())
    assert len(at) == 1


def test_block_with_a_given_input_makes_no_buffer(norms, monkeypatch):
    D = 64
    mix = Mixer(8, D)
    blk = layer.Block(mix, torch.ones(D))
    r, h = torch.zeros(8, D), torch.zeros(8, D, dtype=BF)
    made = count_allocations(monkeypatch)
    blk.forward(r, h=h)
    blk.decode_step(None, r, h=h)
    assert not made and all(s is h for s in mix.seen)


def test_block_says_what_the_mixer_read(norms):
    """Layer.cache_from_prefill wants the input of the layer's last forward: the block has it, its own or the one handed
    in, and decoding leaves it alone."""
    D = 64
    mix = Mixer(8, D)
    blk = layer.Block(mix, torch.ones(D))
    assert blk.h is None
    r = torch.zeros(8, D)
    blk.forward(r)
    own = blk.h
    assert own is mix.seen[-1] and own.shape == (8, D)
    blk.decode_step(None, r)
    assert blk.h is own and mix.seen[-1].data_ptr() != own.data_ptr()
    given = torch.zeros(8, D, dtype=BF)
    blk.forward(r, h=given)
    assert blk.h is given


# ---------------------------------------------------------------- rows of no sequence
FAKE = 1 << 20


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), A.ERR_UNSUPPORTED), (dict(y=None), A.ERR_INVALID_ARG), (dict(y=FAKE + 8), A.ERR_INVALID_ARG),
    (dict(D=60), A.ERR_INVALID_ARG), (dict(D=0), A.ERR_INVALID_ARG), (dict(ldy=56), A.ERR_INVALID_ARG),
    (dict(ldy=68), A.ERR_INVALID_ARG), (dict(seqs=None), A.ERR_INVALID_ARG), (dict(slots=FAKE), A.ERR_INVALID_ARG),
    (dict(seqs=None, slots=FAKE, B=0), A.ERR_INVALID_ARG), (dict(seqs=None, slots=FAKE, B=(1 << 20) + 1), A.ERR_UNSUPPORTED),
    (dict(seqs=A.SeqsT(FAKE, None, None, 0, 2)), A.ERR_INVALID_ARG), (dict(seqs=A.SeqsT(None, None, None, 9, 2)), A.ERR_INVALID_ARG),
    (dict(seqs=A.SeqsT(FAKE, None, None, 9, 1 << 21)), A.ERR_UNSUPPORTED)])
def test_clear_rows_refuses(kw, code):
    a = dict(dtype=A.BF16, y=FAKE, ldy=64, D=64, seqs=A.SeqsT(FAKE, None, None, 16, 2), B=0, slots=None)
    a.update(kw)
    L = A.load()
    assert L.attamba_clear_rows(a["dtype"], a["y"], a["ldy"], a["D"], a["seqs"], a["B"], a["slots"], None) == code
    assert L.attamba_last_error().startswith(b"attamba_clear_rows: ")


def test_clear_rows_takes_no_cpu_tensor():
    with pytest.raises(A.AttambaError, match="CUDA"):
        A.clear_rows(torch.zeros(4, 64), slots=torch.zeros(4, dtype=torch.int32))


class Recorder:
    """attamba's calls as a list of their names, with the rows that clear_rows got."""

    def __init__(self, monkeypatch):
        self.calls = []
        for name in ("proj_gemm", "causal_conv", "conv_step", "selective_scan", "scan_step", "clear_rows"):
            monkeypatch.setattr(A, name, lambda *a, _n=name, **kw: self.calls.append((_n, a, kw)))


def mixer_on_the_cpu(D=64, Di=128, N=16, K=4, rows=8):
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    w = dict(W_in=z(2 * Di, D), W_x=z(Di + 2 * N, Di), W_O=z(D, Di), conv_w=z(Di, K, dt=torch.float32),
             A=z(Di, N, dt=torch.float32))
    return layer.SsmMixer(D, Di, N, K, w, rows, device="cpu")


def test_mixer_clears_rows_of_no_sequence_ahead_of_the_output_product(monkeypatch):
    mix = mixer_on_the_cpu()
    rec = Recorder(monkeypatch)
    state, seqs, slots = mix.new_state(4), object(), torch.zeros(5, dtype=torch.int32)
    names = lambda: [n for n, _, _ in rec.calls]  # noqa: E731
    mix.forward(torch.zeros(7, 64, dtype=BF), seqs, state=state)
    assert names() == ["proj_gemm", "causal_conv", "proj_gemm", "selective_scan", "clear_rows", "proj_gemm"]
    _, a, kw = rec.calls[4]
    assert a[0].data_ptr() == mix.buf["s"].data_ptr() and a[0].shape[0] == 7 and kw["seqs"] is seqs
    assert rec.calls[5][1][0].data_ptr() == a[0].data_ptr()
    rec.calls.clear()
    mix.decode_step(state, torch.zeros(5, 64, dtype=BF), slots=slots)
    assert names() == ["proj_gemm", "conv_step", "proj_gemm", "scan_step", "clear_rows", "proj_gemm"]
    assert rec.calls[4][2]["slots"] is slots and rec.calls[4][1][0].shape[0] == 5
    rec.calls.clear()
    mix.decode_step(state, torch.zeros(4, 64, dtype=BF))          # every row has its state: nothing to clear
    assert "clear_rows" not in names()


# ---------------------------------------------------------------- devices
class Rows:
    """What a device check reads of a tensor."""

    def __init__(self, device, shape=(4, 64)):
        self.device, self.shape, self.dtype = torch.device(device), torch.Size(shape), BF


class Stream:
    def __init__(self, index):
        self.device_index = index


@pytest.mark.parametrize("where,current,stream,match", [
    ("cuda:1", 0, None, "cuda:1 is not the current device"), ("cuda:0", 0, None, "on cuda:0"),
    ("cuda:1", 1, Stream(0), "stream is on cuda:0"), ("cpu", 1, None, "on cpu")])
def test_mixer_and_block_refuse_another_device(monkeypatch, norms, where, current, stream, match):
    """The projections launch on the current device, the other operators on their tensors': a mixer whose buffers are on
    cuda:1 takes tensors and streams of cuda:1 with cuda:1 current, and says so before any call."""
    mix = mixer_on_the_cpu()
    mix.device = torch.device("cuda", 1)
    blk = layer.Block(mix, torch.ones(64))
    rec = Recorder(monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    for call in (lambda: mix.forward(Rows(where), None, stream=stream), lambda: mix.decode_step((None, None), Rows(where), stream=stream),
                 lambda: blk.forward(Rows(where), None, stream=stream), lambda: blk.decode_step((None, None), Rows(where), stream=stream)):
        with pytest.raises(A.AttambaError, match=match):
            call()
    assert not rec.calls and not norms


def test_mixer_runs_where_its_buffers_are(monkeypatch):
    mix = mixer_on_the_cpu()
    mix.device = torch.device("cuda", 1)
    rec = Recorder(monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    mix.decode_step((None, None), Rows("cuda:1"), stream=Stream(1))
    assert rec.calls


def test_block_around_a_layer_refuses_another_device(monkeypatch, norms):
    class Lay(Mixer):
        device = torch.device("cuda", 0)

    blk = layer.Block(Lay(4, 64), torch.ones(64))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(A.AttambaError, match="on cuda:1"):
        blk.forward(Rows("cuda:1"))
    with pytest.raises(A.AttambaError, match="cuda:0 is not the current device"):
        blk.forward(Rows("cuda:0"), h=Rows("cuda:0"))
    assert not norms


@pytest.mark.parametrize("name", ["W_in", "W_x", "W_O", "conv_w", "A", "bias"])
def test_mixer_refuses_weights_on_another_device(name):
    D, Di, N, K = 64, 128, 16, 4
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
    f32 = torch.float32
    w = dict(W_in=z(2 * Di, D), W_x=z(Di + 2 * N, Di), W_O=z(D, Di), conv_w=z(Di, K, dt=f32), A=z(Di, N, dt=f32), bias=z(Di, dt=f32))
    w[name] = w[name].to("meta")
    with pytest.raises(A.AttambaError, match=f"{name} must be on cpu, got meta"):
        layer.SsmMixer(D, Di, N, K, w, 8, device="cpu")


def test_mixer_refuses_buffers_on_another_device():
    with pytest.raises(A.AttambaError, match="buffers"):
        D, Di, N, K = 64, 128, 16, 4
        z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)  # noqa: E731
        f32 = torch.float32
        w = dict(W_in=z(2 * Di, D), W_x=z(Di + 2 * N, Di), W_O=z(D, Di), conv_w=z(Di, K, dt=f32), A=z(Di, N, dt=f32))
        layer.SsmMixer(D, Di, N, K, w, 8, device="cpu", alloc=lambda shape, dt: torch.empty(shape, dtype=dt, device="meta"))


@pytest.mark.parametrize("shape", [(64,), (2, 3, 64)])
def test_block_refuses_a_stream_that_is_not_rows(norms, shape):
    blk = layer.Block(Mixer(8, 64), torch.ones(64))
    for call in (lambda: blk.forward(torch.zeros(shape)), lambda: blk.decode_step(None, torch.zeros(shape))):
        with pytest.raises(A.AttambaError, match=r"r must be \[rows, D\]"):
            call()
    assert not norms


def test_a_refused_call_does_not_spoil_the_block(monkeypatch):
    """A stream of a wrong width or device makes no buffer that later calls would be handed."""
    D = 64
    monkeypatch.setattr(A, "block_norm", lambda y, res, res_out=None, h=None, **kw: None)
    mix = Mixer(16, D)
    blk = layer.Block(mix, torch.ones(D))
    for bad in (torch.zeros(16, 2 * D), torch.zeros(16, D, device="meta")):
        blk.decode_step(None, bad)               # the library refuses these; here the recorders take them
        blk.decode_step(None, torch.zeros(5, D))
        assert mix.seen[-1].shape == (5, D) and mix.seen[-1].device.type == "cpu"
