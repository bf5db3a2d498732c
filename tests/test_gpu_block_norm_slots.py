"""The gradients of the slots' gates (eidm_block_norm_backward) where almost
all of a sum cancels, on the GPU against the formulas in 64 bits."""
import pytest
import torch

from test_gpu_block_norm import EXACT, Norm, formula, gradients

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,hidden", [(9, 2048), (5, 4095), (9, 4100), (300, 5003), (3, 12292), (2, 20001)])
@pytest.mark.parametrize("gate", ["none", "token"])
def test_the_gate_of_a_single_normed_slot(lib, m, hidden, gate):
    """The norm takes the slot's gate out again but for eps: its gradient is what d_z . y leaves, some eps of its terms."""
    c = Norm(lib, "bf16", "f32", m, hidden, 1, True, True, gate, True)
    c.slot_gates += 0.5
    rows = c.block(c.leaves()).to(c.x.dtype)
    got = gradients(c, rows)["d_slot_gates"].double()
    want, d_stream, z = formula(c, rows)
    want = want["d_slot_gates"]
    scale = 1 + float(d_stream.abs().max()) * (1 + float(z.abs().max()))
    # half a step of the result, and the 64-bit sum of rounded 64-bit terms
    bound = want.abs() * 2.0 ** -24 * (1 + 2.0 ** -10) + EXACT * scale * 50
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())


@pytest.mark.parametrize("hidden", [600, 5003, 8192, 12292, 13000])
@pytest.mark.parametrize("top_k,slot", [(4, 3), (6, 0), (6, 5), (11, 9)])
def test_the_gate_of_the_only_slot_that_counts(lib, hidden, top_k, slot):
    """The same where the other slots' gates are zero; theirs have ordinary gradients."""
    c = Norm(lib, "f32", "bf16", 7, hidden, top_k, True, True, "channel", True)
    c.slot_gates[:, :] = 0
    c.slot_gates[:, slot] = 0.75
    rows = c.block(c.leaves()).to(c.x.dtype)
    got = gradients(c, rows)["d_slot_gates"].double()
    want, d_stream, z = formula(c, rows)
    want = want["d_slot_gates"]
    scale = 1 + float(d_stream.abs().max()) * (1 + float(z.abs().max()))
    bound = want.abs() * 2.0 ** -24 * (1 + 2.0 ** -10) + EXACT * scale * 50
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
