"""Widths and lengths whose kernels no other test of the 8-bit block reaches:
experts between the powers of two, rows of every units-a-thread form."""
import numpy as np
import pytest
import torch

import i8_cases as I
from expert_id_matmul_amd import binding as B
from test_gpu_balance import DEPTH, SCORE, SLOPE, ULP, Case
from test_gpu_block_norm import EXACT, Norm, close, columns, formula, gradients
from test_gpu_ffn_i8 import Ffn
from test_gpu_i8 import DTYPES, quantize

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,experts,top_k,seqs", [(90, 300, 8, 4), (200, 512, 8, 7), (3000, 511, 4, None), (70, 257, 3, 3),
                                                  (50, 1024, 6, 3), (40, 1500, 8, 2)])
def test_balance_between_the_widths(lib, m, experts, top_k, seqs):
    c = Case(lib, m, experts, top_k, seqs, True, 1.0)
    counts, mean, loss = c.forward()
    want_counts, want_mean, want_loss, want, size = c.formula()
    assert torch.equal(counts.view(c.n, c.e).long(), want_counts)
    bound = (2 * SCORE + DEPTH + 3 + c.m) * ULP
    assert ((mean.view(c.n, c.e).double() - want_mean).abs() <= bound * want_mean + 1e-30).all()
    assert abs(float(loss) - want_loss) <= bound * want_loss + 1e-30
    off = (c.backward(counts).double() - want).abs()
    assert (off <= (4 * SCORE + 3 * DEPTH + SLOPE + 8) * ULP * size + 1e-30).all()


@pytest.mark.parametrize("experts", [65, 100, 200, 400, 512, 700, 1200, 2048])
@pytest.mark.parametrize("m,top_k", [(1, 8), (3, 4)])
def test_the_ffn_of_a_few_tokens_at_any_number_of_experts(lib, experts, m, top_k):
    c = Ffn(lib, m, 96, 40, top_k, experts, True, True)
    got = c.result(B.DIRECT)
    assert lib.last_dispatch().kernels() == ["i8_gate_up_one", "i8_down_rows"]
    c.check(got, I.ffn(c.d, top_k, True))
    np.testing.assert_array_equal(got, c.result(B.GROUPED))


# more rows than the kernels have blocks for in one turn, or rows a block takes together
@pytest.mark.parametrize("m,hidden", [(5000, 333), (5000, 500), (2100, 1000), (1100, 515), (2100, 1023), (1100, 1500),
                                      (600, 3001), (300, 6000)])
@pytest.mark.parametrize("gate", ["token", "channel"])
def test_norms_of_many_rows(lib, m, hidden, gate):
    c = Norm(lib, "bf16", "bf16", m, hidden, 2, True, True, gate, True)
    out, normed, q, q_scales = c.forward(q=True)
    close(out, c.block(c.leaves()), c.dtype, "out")
    close(normed, c.normed(out.double(), c.w_pre.double()), "f32", "normed")
    want_q, scales = I.quantize(normed.numpy())
    I.same(q_scales, scales)
    np.testing.assert_array_equal(q.numpy(), want_q)
    got = gradients(c, out)
    want, d_stream, z = formula(c, out)
    scale = 1 + float(d_stream.abs().max()) * (1 + float(z.abs().max()))
    for n in ("d_x", "d_z"):
        off = (got[n].double() - want[n]).abs()
        assert (off <= want[n].abs() * 2.0 ** -24 * (1 + 2.0 ** -10) + EXACT * scale * 50).all(), n
    terms = (want["d_z"].unsqueeze(1) * c.y.double().view(c.m, c.k, c.h)).abs().sum(2)
    assert ((got["d_slot_gates"].double() - want["d_slot_gates"]).abs() <= terms * 2.0 ** -23 + EXACT * scale * 50).all()
    n = z / torch.sqrt((z * z).mean(1, keepdim=True) + c.eps)
    g = c.gate.double()[:, None] if gate == "token" else c.gate.double()
    columns(got["d_w_post"], want["d_w_post"], d_stream * g * n, "d_w_post")
    r = out.double()
    columns(got["d_w_pre"], want["d_w_pre"], c.d_normed.double() * r / torch.sqrt((r * r).mean(1, keepdim=True) + c.eps),
            "d_w_pre")
    if gate == "channel":
        columns(got["d_gate"], want["d_gate"], d_stream * n * c.w_post.double(), "d_gate")
    else:
        off = (got["d_gate"].double() - want["d_gate"]).abs()
        assert (off <= want["d_gate"].abs() * 2.0 ** -23 + EXACT * scale * c.h * 50).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,k", [(9000, 512), (9000, 1024), (9000, 2048), (9000, 1500), (5, 4096), (70, 4000), (9000, 4096)])
def test_rows_of_every_form(lib, dtype, rows, k):
    g = torch.Generator().manual_seed(rows + k)
    x = (torch.randn(rows, k, generator=g) * torch.rand(rows, 1, generator=g) * 3).to(DTYPES[dtype])
    q, s = quantize(lib, x.cuda())
    want_q, want_s = I.quantize(x.float().numpy())
    I.same(s, want_s)
    np.testing.assert_array_equal(q, want_q)
