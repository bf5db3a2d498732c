"""The expert FFN in 8 bits (eidm_moe_ffn_i8) of more tokens than a launch of
2^32 threads has blocks for, one to quantise each and one to route four."""
import pytest
import torch

from expert_id_matmul_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "eight_bits"])
def test_many_tokens(lib, eight):
    """Each token's results depend on no other: those of a few tokens by themselves have the same bits."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("not 12 GiB of device memory free")
    torch.manual_seed(4)
    m, hidden, inter, experts = 18_000_001, 20, 16, 2
    w = [torch.randint(-127, 128, s, dtype=torch.int8, device="cuda")
         for s in ((experts, inter, hidden), (experts, inter, hidden), (experts, hidden, inter))]
    scales = [0.02 * torch.rand(experts, n, device="cuda") for n in (inter, inter, hidden)]
    x, logits = torch.randn(m, hidden, device="cuda"), torch.randn(m, experts, device="cuda")
    x_scales = None
    if eight:
        x, x_scales = torch.randint(-127, 128, (m, hidden), dtype=torch.int8, device="cuda"), 0.02 * torch.rand(m, device="cuda")

    def run(route, lo, hi):
        n = hi - lo
        shape = B.make_ffn_i8_shape(n, hidden, inter, 1, experts)
        ids, gates = torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda")
        out = torch.full((n, hidden), float("nan"), device="cuda")
        scratch = torch.empty(lib.moe_ffn_i8_scratch_bytes(shape), dtype=torch.uint8, device="cuda")
        lib.moe_ffn_i8(shape, route, w[0], scales[0], w[1], scales[1], w[2], scales[2], x[lo:hi],
                       None if x_scales is None else x_scales[lo:hi], logits[lo:hi], None, ids, gates, out, scratch,
                       renormalize=False)
        return ids, gates, out

    want = run(B.DIRECT, 0, m)
    assert not any(torch.isnan(t).any() for t in want[1:])
    for a, b in zip(want, run(B.GROUPED, 0, m)):
        assert torch.equal(a, b)
    for lo in (0, m // 3, m // 2 - 7, m - 1000):
        for a, b in zip(run(B.DIRECT, lo, lo + 1000), want):
            assert torch.equal(a, b[lo:lo + 1000])
