"""GPU: the recurrence's gates are as accurate as the interface states, and its chain of states over many groups of
chunks agrees with the recurrence step by step."""
import pytest
import torch

from stacked_lstm_forward_amd import block

from .block_reference import FLUSH, W, glr, within
from .test_gpu_block import DEV, DT, Make, glr_check, lengths_of, spoil
from .test_gpu_block_tanh import every_bf16

pytestmark = pytest.mark.gpu


def gates(f):
    """a and 1 - a of f [B, 1, 64], in fp32: the state 1 without a candidate, and no state with a candidate of 1."""
    B = f.shape[0]
    zero, one = torch.zeros_like(f), torch.ones_like(f)
    a = block.prepare_glr(f, zero, c0=torch.ones(B, 64, device=DEV))
    a.forward()
    s = block.prepare_glr(f, one)
    s.forward()
    return a.cT, s.cT


def test_gates_of_every_bf16_value():
    f = every_bf16(2.0 ** -40)
    a, s = gates(f.to(DEV))
    x = f[:, 0].double()
    rel = (6 + 1.3 * x.abs()) * W
    for got, want in ((a, torch.sigmoid(x)), (s, torch.sigmoid(-x))):
        within(got, (want, rel * want + FLUSH), "gate")


def test_gates_of_fp32_values():
    g = torch.Generator().manual_seed(3)
    f = torch.cat((torch.rand(500, 1, 64, generator=g) * 240 - 120, torch.randn(500, 1, 64, generator=g),
                   torch.randn(100, 1, 64, generator=g) * 1e-6))
    a, s = gates(f.to(DEV))
    x = f[:, 0].double()
    for got, want in ((a, torch.sigmoid(x)), (s, torch.sigmoid(-x))):
        within(got, (want, 7 * W * want + FLUSH), "gate")


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("bias,by", [(-12.0, 3.0), (12.0, 3.0), (0.0, 30.0)])
def test_glr_shut_and_open_bf16_gates(bias, by, types):
    glr_check(2, 300, 40, types, bias=bias, by=by, seed=3)


# (type, channels, steps): more than 17 chunks forwards (of 256, 512 and 512 steps), so that the states behind two
# groups of eight are used; backwards more
LONG = [("bf16", 64, 17 * 256 + 100), ("bf16", 24, 17 * 512 + 77), ("f32", 4, 17 * 512 + 300)]


@pytest.mark.parametrize("grads", ["f32", "same"])
@pytest.mark.parametrize("dtype,H,T", LONG, ids=str)
def test_states_across_groups_of_chunks(dtype, H, T, grads):
    grads = dtype if grads == "same" else grads
    m = Make(5, T, "tbh", H)
    # long memories: gates so far open that a state outlasts a group
    f, u, o = m.seq(H, dtype, 1.0, 8.0), m.seq(H, dtype), m.seq(H, dtype)
    c0, dy, dcT = m.flat(5, H), m.seq(H, grads), m.flat(5, H)
    n = lengths_of(T, [T, 8 * 512 + 1, 16 * 256, 3, 0])
    for t in (f, u, o, dy):
        spoil(t, n)
    p = block.prepare_glr(f, u, o, c0=c0, lengths=n, train=True, grad_dtype=DT[grads])
    p.forward()
    p.backward(dy, dcT)
    want = glr(f, u, o, c0, n, False, dy, dcT)
    for k, v in want.items():
        within(getattr(p, k), v, k)
