"""examples/hybrid_serving.py as a whole: the logits of tokens decoded one by one
are those of the same tokens prefilled at once, and what a server can get wrong
between its calls shows.

Bound: one block of three delta-rule layers and an attention layer. A layer's
output carries a few roundings of 2^-9 (inputs, weights, outputs, projection),
2^-8 of its size in all; a later layer passes an error on with a factor of about
2 (its input and its own output both move), errors add up as independent ones:
2^-8 sqrt(1 + 4 + 16 + 64) = 3.6e-2 per token and vector of logits. A mistake in
the bookkeeping has to show with twice that in some token.
"""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

FILE = Path(__file__).resolve().parents[1] / "examples" / "hybrid_serving.py"
BOUND = 3.6e-2


@pytest.fixture()
def example():
    spec = importlib.util.spec_from_file_location("hybrid_serving", FILE)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def apart(example, lengths, **kw):
    stepped, once = example.serve(lengths, blocks=1, **kw)
    return (stepped - once).norm(dim=-1) / once.norm(dim=-1)


@pytest.mark.parametrize("lengths,chunk,steps", [((15, 3), 8, 4),
                                                 ((70, 1, 200, 33), 64, 12)])
def test_decoding_gives_the_logits_of_a_prefill(lib, cuda_device, example,
                                                lengths, chunk, steps):
    off = apart(example, lengths, chunk=chunk, steps=steps)
    assert off.max() <= BOUND, off.max()


def short_lengths(server):
    """Every decoded token stands one place too early."""
    grow = server._grow

    def patched(self, new):
        grow(self, new)
        if set(new) == {1}:
            self.lens -= 1
    server._grow = patched


def shared_pages(server):
    """A page taken while decoding is another request's."""
    grow = server._grow

    def patched(self, new):
        count = list(self.pages.count)
        grow(self, new)
        if set(new) == {1} and self.pages.count[0] > count[0]:
            self.pages.table[0, count[0]] = self.pages.table[1, 0]
    server._grow = patched


def dropped_states(server):
    """Decoding starts from zero states."""
    decode = server.decode

    def patched(self, tokens):
        if not getattr(self, "dropped", False):
            self.dropped = True
            self.states = [None if s is None else torch.zeros_like(s)
                           for s in self.states]
        return decode(self, tokens)
    server.decode = patched


@pytest.mark.parametrize("mistake", [short_lengths, shared_pages, dropped_states])
def test_mistakes_show(lib, cuda_device, example, mistake):
    mistake(example.HybridServer)
    off = apart(example, (15, 3), chunk=8, steps=4)
    assert off.max() > 2 * BOUND, off.max()
