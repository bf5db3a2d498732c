"""The router's gradient and balance loss at the ends of the scores' range and
of the calls' sizes, on the GPU against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from expert_id_matmul_amd import binding as B
from test_gpu_balance import DEPTH, SCORE, SLOPE, ULP, Case
from test_gpu_ffn_i8 import Ffn

pytestmark = pytest.mark.gpu

# of a gate's gradient through renormalised gates: a gate is a score over a sum of them (2 * SCORE + 8), the differences
# of d_gates 1, their weighted sum 8, the factor score * (1 - score) / sum at most SCORE + 2 * SLOPE, four steps between
GATES = 2 * (2 * SCORE + 8) + SCORE + 2 * SLOPE + 16


def chosen(c, logits):
    c.logits = logits
    c.ids = torch.topk(logits, c.k, dim=1).indices.int()
    return c


def near(got, want, bound):
    off = (got.double() - want).abs()
    assert (off <= bound).all(), float((off / bound).max())


def test_gates_of_tiny_scores_have_their_gradient(lib):
    """Renormalised gates are ratios: they and their gradient are of order one however small the scores."""
    c = Case(lib, 64, 40, 4, None, True, 1.0)
    g = torch.Generator().manual_seed(8)
    least = torch.rand(64, 1, generator=g) * 80 + 20  # each token's largest logit from -20 down to -100
    chosen(c, (-least - 3 * torch.rand(64, 40, generator=g)).clamp(min=-103.5))
    c.logits[::5, ::3] -= 60  # beside experts far below
    chosen(c, c.logits)
    got = c.backward(c.forward()[0], loss=False)
    _, _, _, want, size = c.formula(loss=False)
    assert want.abs().max(1).values.min() > 1e-3
    near(got, want, GATES * ULP * size + 1e-30)


def test_gates_without_a_score_have_no_gradient(lib):
    """The router's scores are f32: below about -103.97 they are 0, and where all picks' are, no gate is a number."""
    c = Case(lib, 12, 40, 4, None, True, 1.0)
    c.logits[3], c.logits[5], c.logits[7] = -104.0, float("-inf"), -1e30
    c.logits[8] = -103.9
    chosen(c, c.logits)
    got = c.backward(c.forward()[0], loss=False)
    assert torch.isfinite(got).all() and (got[[3, 5, 7]] == 0).all()
    d = c.d_gates[8].double()
    near(got[8, c.ids[8].long()], (d - d.mean()) / 4, GATES * ULP * d.abs().sum())


def test_a_pick_that_is_no_number_stays_in_its_token(lib):
    c = Case(lib, 12, 40, 4, None, True, 1.0)
    counts = c.forward()[0]
    want = c.backward(counts)
    for value in (float("nan"), -90.0):
        other = -90.0 if value != value else float("nan")
        c.logits[6, c.ids[6, :3].long()] = value
        c.logits[6, c.ids[6, 3].long()] = other
        got = c.backward(counts)
        assert torch.isnan(got[6, c.ids[6].long()]).all()
        rest = torch.arange(12) != 6
        assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("m,hidden", [(1, 96), (12, 96), (12, 9000)], ids=["one", "one_launch", "start"])
@pytest.mark.parametrize("renormalize", [True, False], ids=["renormalised", "as_they_are"])
def test_a_token_of_masked_experts_alone(lib, m, hidden, renormalize):
    """No score: NaN gates and a row of NaN where the gates are renormalised, zeros where not, and no other row's matter;
    the gradient through its gates is zero."""
    c = Ffn(lib, m, hidden, 64, 3, 6, True, renormalize)
    clean = {r: c.result(r) for r in (B.DIRECT, B.GROUPED)}
    masked = m // 2
    for value in (float("-inf"), -104.0):
        c.logits[masked] = value
        for r, want in clean.items():
            got = c.result(r)
            assert np.isnan(got[masked]).all() if renormalize else (got[masked] == 0).all()
            np.testing.assert_array_equal(np.delete(got, masked, 0), np.delete(want, masked, 0))
            assert (c.ids.cpu() >= 0).all() and (c.ids.cpu() < 6).all()
        d = torch.full((m, 6), float("nan"), device="cuda")
        lib.route_backward(B.make_balance_shape(m, 6, 3), c.logits, c.ids, None, torch.ones(1, 6, dtype=torch.int32).cuda(),
                           torch.ones(m, 3).cuda(), None, d, renormalize=renormalize)
        assert (d[masked] == 0).all() and torch.isfinite(d).all()


def test_a_gate_beside_tiny_ones_has_its_gradient(lib):
    """d_gates[j] less the weighted mean of them all, where one gate has nearly all the weight: the sum of the differences
    from that gate's, in which nothing cancels."""
    c = Case(lib, 64, 40, 4, None, True, 1.0)
    g = torch.Generator().manual_seed(9)
    logits = -14 - 4 * torch.rand(64, 40, generator=g)
    logits[torch.arange(64), torch.randint(0, 40, (64,), generator=g)] = 2 * torch.randn(64, generator=g)
    chosen(c, logits)
    c.ids = c.ids[:, torch.randperm(4, generator=g)].contiguous()  # with a selection bias the largest score is anywhere
    got = c.backward(c.forward()[0], loss=False)
    _, _, _, want, _ = c.formula(loss=False)
    at, d = c.ids.long(), c.d_gates.double()
    s = torch.sigmoid(torch.gather(c.logits.double(), 1, at))
    gate, top = s / s.sum(1, keepdim=True), s.argmax(1, keepdim=True)
    off = (d - torch.gather(d, 1, top)).abs()
    size = torch.zeros(64, 40, dtype=torch.float64).scatter_(1, at, gate * (1 - s) * (off + (gate * off).sum(1, keepdim=True)))
    near(got, want, GATES * ULP * size)


@pytest.mark.parametrize("experts", [40, 700])
def test_probabilities_of_tiny_scores(lib, experts):
    """A token whose largest score is near the smallest number has probabilities like any other."""
    c = Case(lib, 50, experts, 3, [0, 20, 50], True, 1.0)
    g = torch.Generator().manual_seed(10)
    logits = -84 - 8 * torch.rand(50, experts, generator=g)
    logits[::2] += 55 * torch.rand(25, 1, generator=g)
    chosen(c, logits)
    assert (c.logits.max(1).values > -87).all() and (c.logits.min(1).values < -87.4).any()
    counts, mean, loss = c.forward()
    _, want_mean, want_loss, want, size = c.formula(gates=False)
    bound = (2 * SCORE + DEPTH + 3 + c.m) * ULP
    near(mean.view(2, -1), want_mean, bound * want_mean)
    assert abs(float(loss) - want_loss) <= bound * want_loss
    near(c.backward(counts, gates=False), want, (4 * SCORE + 3 * DEPTH + SLOPE + 8) * ULP * size)


def test_more_than_2_to_the_30_tokens(lib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 20 * 2 ** 30:
        pytest.skip("not 20 GiB of device memory free")
    m = 2 ** 30 + 12345
    torch.manual_seed(3)
    logits, d_gates = torch.empty(m, 1, device="cuda").normal_(), torch.empty(m, 1, device="cuda").normal_()
    ids, counts = torch.zeros(m, 1, dtype=torch.int32, device="cuda"), torch.full((1, 1), m, dtype=torch.int32, device="cuda")
    got = torch.full((m, 1), float("nan"), device="cuda")
    lib.route_backward(B.make_balance_shape(m, 1, 1), logits, ids, None, counts, d_gates, None, got, renormalize=False)
    for lo in range(0, m, 1 << 26):
        s = torch.sigmoid(logits[lo:lo + (1 << 26)].double())
        want = d_gates[lo:lo + (1 << 26)].double() * s * torch.sigmoid(-logits[lo:lo + (1 << 26)].double())
        assert ((got[lo:lo + (1 << 26)].double() - want).abs() <= (SLOPE + 2) * ULP * want.abs() + 1e-30).all()


@pytest.mark.parametrize("uneven", [0, 1, 40])
@pytest.mark.parametrize("experts", [16, 200])
def test_even_loads_leave_no_rounding(lib, experts, uneven):
    """Probabilities add up to one: the loss's gradient is of the loads' distances from one, none with even picks."""
    c = Case(lib, 400, experts, 4, [0, 400], True, 1.0)
    c.ids = torch.arange(1600).remainder(experts).view(400, 4).int()
    c.ids.view(-1)[:uneven] = (c.ids.view(-1)[:uneven] + 3) // 2
    counts = c.forward()[0]
    got = c.backward(counts, gates=False)
    _, _, _, want, _ = c.formula(gates=False)
    if not uneven:
        assert (got == 0).all()
    s = torch.sigmoid(c.logits.double())
    p = s / s.sum(1, keepdim=True)
    off = (counts.double() * experts / 1600 - 1).abs()
    size = float(c.d_loss) / 400 * (off + (p * off).sum(1, keepdim=True)) * p * (1 - s)
    near(got, want, (4 * SCORE + 3 * DEPTH + SLOPE + 8) * ULP * size + 1e-18)


@pytest.mark.parametrize("tokens,experts,top_k", [(7 * 49, 49, 3), (6 * 110, 110, 7), (29 * 13, 13, 11), (23 * 6, 18, 3)])
def test_even_loads_of_any_size_have_no_gradient(lib, tokens, experts, top_k):
    c = Case(lib, tokens, experts, top_k, [0, tokens], True, 1.0)
    c.ids = torch.arange(tokens * top_k).remainder(experts).view(tokens, top_k).int()
    counts = c.forward()[0]
    assert (counts == tokens * top_k // experts).all()
    assert (c.backward(counts, gates=False) == 0).all()
