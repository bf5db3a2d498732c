"""Which kernels eidm_lora_linear takes, by the dispatch receipt, and their
bits: the shared projection's forms against eidm_matmul_id's Direct route, the
adapters' forms against the documented order."""
import pytest
import torch

from expert_id_matmul_amd import binding as B
from expert_id_matmul_amd import workloads as W
from helpers import check_guarded, poisoned_output

pytestmark = pytest.mark.gpu

BF, HF, FL = W.DT_BF16, W.DT_F16, W.DT_F32
TORCH = {FL: torch.float32, HF: torch.float16, BF: torch.bfloat16}


def projection(lib, dtype, m, n, k, arith, a_dtype=None):
    """lora_linear's shared projection (no row has an adapter), compared with
    eidm_matmul_id's Direct route bit for bit; -> the call's receipt."""
    a_dtype = dtype if a_dtype is None else a_dtype
    g = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.randn(m, k, generator=g, device="cuda")
    w = torch.empty(n, k, device="cuda", dtype=TORCH[dtype])
    w.normal_(0, k ** -0.5, generator=g)
    a, b = (torch.zeros(1, *z, device="cuda", dtype=TORCH[a_dtype]) for z in ((4, k), (n, 4)))
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    shape = B.make_lora_shape(dtype, a_dtype, m, n, k, 1, 4, arith=arith)
    scratch = torch.full((lib.lora_linear_scratch_bytes(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    out = poisoned_output(m * n)
    lib.lora_linear(shape, w, None, a, b, None, None, x, ids, out, scratch)
    receipt = lib.last_dispatch()
    want = torch.empty(m, n, device="cuda")
    s = B.make_shape(dtype, m, n, k, 1, 1, n * k * W.DTYPE_SIZE[dtype], arith=arith)
    ds = torch.empty(max(1, lib.query(s, B.DIRECT).scratch_bytes), dtype=torch.uint8, device="cuda")
    lib.matmul_id(s, B.DIRECT, w, x, torch.zeros(m, 1, dtype=torch.int32, device="cuda"), want, ds)
    torch.cuda.synchronize()
    assert torch.equal(out[: m * n].view(m, n).view(torch.int32), want.view(torch.int32))
    check_guarded(out, m * n)
    return receipt


@pytest.mark.parametrize("m,n,k,dense", [
    (1, 16384, 4096, False), (16, 16384, 4096, False), (64, 16384, 4096, False), (1, 32768, 4096, False),
    (16, 32768, 4096, False), (1, 32768, 512, False), (32, 65536, 512, False), (96, 16384, 4096, False),
    (12000, 200, 4096, False), (64, 65536, 512, True), (129, 16384, 4096, True), (96, 16384, 512, True),
    (1500, 1500, 4096, True), (1024, 2048, 1024, True)])
def test_dense_split16_tiles_only_where_they_are_the_faster_ones(lib, m, n, k, dense):
    """128 x 128 tiles serve many rows; a few rows of a wide projection, or many
    of a narrow one, take eidm_matmul_id's kernels (measured at these sizes)."""
    print(f"[case] {m} {n} {k}", flush=True)
    assert ("dense_split16" in projection(lib, BF, m, n, k, B.ARITH_SPLIT16).kernels()) == dense


@pytest.mark.parametrize("dtype,m,n,k", [(BF, 1, 24592, 520), (HF, 1, 40007, 260), (FL, 1, 33000, 200), (BF, 2, 32768, 1024),
                                         (BF, 4, 65536, 512), (HF, 3, 50001, 129), (FL, 4, 30011, 140)])
def test_up_to_four_rows_are_staged_at_any_width(lib, dtype, m, n, k):
    """A vocabulary's width for a few rows: one launch with the adapters'
    shrink, then the expand."""
    print(f"[case] {dtype} {m} {n} {k}", flush=True)
    assert projection(lib, dtype, m, n, k, B.ARITH_F32).kernels() == ["lora_base", "lora_expand"]


@pytest.mark.parametrize("dtype,m,n,k", [(BF, 2048, 16, 264), (HF, 2048, 64, 520), (FL, 2047, 30, 100), (BF, 1500, 144, 136),
                                         (BF, 8000, 32, 128), (HF, 5, 1003, 300)])
def test_projection_tiles_are_spread_over_all_xcds(lib, dtype, m, n, k):
    """As many blocks as tiles, rounded up to the eight XCDs: none of them idle
    beside others with several turns (2048 x 64 x 4096 took 83 us so, 41 now)."""
    receipt = projection(lib, dtype, m, n, k, B.ARITH_F32, BF if dtype == FL else FL)
    assert receipt.kernels()[-3:] == ["lora_shrink", "lora_base", "lora_expand"]
    tiles = {(-(-m // (16 * r))) * (-(-n // (16 * c))) for r, c in ((1, 1), (1, 2), (2, 2), (2, 3))}
    assert receipt.launches[receipt.recorded - 2].grid in {-(-t // 8) * 8 for t in tiles}
