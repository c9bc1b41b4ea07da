"""CPU: a clipping problem's tensors are looked at before every call, not only their addresses."""
import pytest
import torch

from stacked_lstm_forward_amd import block
from stacked_lstm_forward_amd.held import Held

CHANGES = [
    ("fewer", lambda x: x[:50]), ("more", lambda x: torch.empty(0).set_(x.untyped_storage(), 0, (150,))),
    ("other type", lambda x: x.view(torch.bfloat16)), ("other type, as many", lambda x: x.view(torch.bfloat16)[:100]),
    ("strided", lambda x: torch.empty(0).set_(x.untyped_storage(), 0, (100,), (2,))), ("none", lambda x: x[:0]),
]


def flat():
    return torch.zeros(300)[:100]


@pytest.mark.parametrize("which", ["tensor", "output", "both"])
@pytest.mark.parametrize("name,change", CHANGES, ids=[c[0] for c in CHANGES])
def test_a_tensor_changed_at_its_address_is_refused(name, change, which):
    t, out = flat(), flat()
    p = block.prepare_clip([torch.zeros(7), t], 1.0, out=None if which == "both" else [torch.zeros(7), out])
    x = out if which == "output" else t
    first, at = x.data, x.data_ptr()
    x.data = change(first)
    assert x.data_ptr() == at or x.numel() == 0
    for _ in range(2):
        with pytest.raises(ValueError, match="1: no longer what the problem was made for"):
            p.run()
    x.data = first
    with pytest.raises(ValueError, match="the kernels run on a GPU"):  # (nothing else is wrong with it)
        p.run()


def test_resized_in_place():
    t = torch.zeros(100)
    p = block.prepare_clip([t], 1.0)
    t.resize_(60)
    with pytest.raises(ValueError, match="no longer"):
        p.run()
    t.resize_(100)
    with pytest.raises(ValueError, match="the kernels run on a GPU"):
        p.run()


def test_other_memory_is_followed():
    t, other = torch.zeros(100), torch.zeros(100)
    p = block.prepare_clip([t], 1.0)
    t.data = other
    assert p._moved() and p._list[0].src == p._list[0].dst == other.data_ptr()
    assert not p._moved()
    t.data = torch.zeros(10, 10)  # as many values in the same order
    assert p._moved() and p._list[0].src == t.data_ptr()
    out = torch.zeros(100)
    q = block.prepare_clip([other], 1.0, out=[out])
    out.data = other[50:].new_zeros(100)
    assert q._moved() and q._list[0].dst == out.data_ptr() and q._list[0].src == other.data_ptr()
    out.data = torch.cat((other, other))[50:150]
    assert q._moved()
    both = torch.zeros(150)
    a, b = both[:100], torch.zeros(100)
    r = block.prepare_clip([a], 1.0, out=[b])
    b.data = both[50:]  # now over the other's end
    for _ in range(2):
        with pytest.raises(ValueError, match="overlap"):
            r.run()


def test_held():
    x, y = torch.zeros(4, 5), torch.zeros(3, dtype=torch.bfloat16)
    h = Held((x, y))
    assert h.same()
    x.add_(1)
    assert h.same()
    x.t_()
    assert not h.same()
    h.read()
    assert h.same()
    for bad in ((x, None), (3,), (x, [y])):
        with pytest.raises(TypeError):
            Held(bad)
    assert Held(()).same()
