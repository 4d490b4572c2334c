"""What svdq_linear_chain takes for a linear and what for a step between linears (the linears
here only note their calls)."""

from types import SimpleNamespace

import torch

import rank_bit_residual_b200 as rb


def test_entries_of_a_chain(monkeypatch):
    seen = []

    def linear(w, x, **kw):
        seen.append((w, kw["bias"], kw["out"], kw["pdl"]))
        return x + w.add

    monkeypatch.setattr(rb, "svdq_linear", linear)

    class Callable(rb.PreparedWeight):
        """A prepared weight stays one, whatever else it can do."""
        add = 100

        def __init__(self):
            pass

        def __call__(self, x):
            raise AssertionError("called")

    alike = SimpleNamespace(add=1)           # the attributes of a prepared weight in another object
    own = Callable()
    x, bias, out = torch.zeros(2), torch.ones(1), torch.ones(2)
    y = rb.svdq_linear_chain([alike, lambda t: t * 10, own], x, biases=[bias, None, None], outs=[None, None, out])
    assert torch.equal(y, torch.full((2,), 110.0))
    assert [w for w, *_ in seen] == [alike, own]
    assert [rest for _, *rest in seen] == [[bias, None, False], [None, out, True]]
