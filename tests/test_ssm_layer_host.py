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
