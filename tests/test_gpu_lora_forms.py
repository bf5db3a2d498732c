"""Which kernels eidm_lora_linear takes, by the dispatch receipt, and their
bits: the shared projection's forms against eidm_matmul_id's Direct route, the
adapters' forms against the documented order."""
import numpy as np
import pytest
import torch

from expert_id_matmul_amd import binding as B
from expert_id_matmul_amd import workloads as W
from helpers import check_guarded, poisoned_output
from lora_cases import Lora, base_bits, documented, inputs
from test_gpu_lora import Call, same_bits

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


@pytest.mark.parametrize("dtype,m,n,k", [(BF, 900, 1003, 137), (HF, 1031, 2000, 264), (FL, 512, 2048, 300), (BF, 512, 4096, 1024),
                                         (BF, 5, 131000, 64), (HF, 16384, 75, 130), (FL, 2048, 2040, 65)])
def test_many_small_tiles_of_short_products(lib, dtype, m, n, k):
    """Up to 16 tiles of 32 x 32 a compute unit where k is short (up to twice as
    fast as the gathered kernels with their map)."""
    print(f"[case] {dtype} {m} {n} {k}", flush=True)
    assert "lora_base" in projection(lib, dtype, m, n, k, B.ARITH_F32).kernels()


@pytest.mark.parametrize("dtype,m,n,k,a_dtype", [(BF, 4100, 1030, 137, None), (HF, 4200, 1000, 264, FL), (FL, 512, 2048, 6001, None),
                                                 (BF, 512, 4096, 3000, None), (BF, 5, 131104, 64, None)])
def test_projections_beyond_the_small_tiles(lib, dtype, m, n, k, a_dtype):
    """Long products of more than three 32 x 32 tiles a compute unit, the ordinary
    prompt chunk: the F32 order through eidm_matmul_id, its ids written by the shrink."""
    print(f"[case] {dtype} {m} {n} {k}", flush=True)
    kernels = projection(lib, dtype, m, n, k, B.ARITH_F32, a_dtype).kernels()
    assert "lora_shrink" in kernels and kernels[-1] == "lora_expand" and "lora_base" not in kernels
    assert kernels[-2].startswith("grouped")


SORTED = ["lora_shrink", "lora_expand"]  # behind a map


@pytest.mark.parametrize("p", [Lora("chunk", BF, BF, 1300, 1024, 264, 6, 16, runs=4),
                               Lora("chunk_odd", HF, FL, 1900, 1003, 139, 9, 11, runs=7, pad=3),
                               Lora("chunk_f32", FL, FL, 1290, 611, 300, 4, 33, runs=5),
                               Lora("adapters_65", BF, BF, 1400, 700, 628, 65, 16),
                               Lora("adapters_130", BF, HF, 1200, 577, 431, 130, 33, pad=1),
                               Lora("adapters_300_given", FL, BF, 1200, 830, 996, 300, 24, given=True),
                               Lora("most_adapters", BF, BF, 4000, 250, 900, 2048, 40),
                               Lora("most_adapters_f32", FL, FL, 11000, 233, 600, 2048, 9, given=True),
                               Lora("one_adapter_of_many", BF, BF, 1400, 300, 500, 500, 64, runs=1, none=0.0),
                               Lora("two_of_many", HF, HF, 1100, 270, 588, 200, 48, runs=3, given=True),
                               Lora("long_k_f32", FL, FL, 37, 63, 16300, 6, 19),
                               Lora("long_k_odd", HF, BF, 70, 77, 16301, 5, 41, pad=1),
                               Lora("long_k_most_ranks", BF, BF, 50, 130, 16264, 3, 256, given=True, ranks=False),
                               Lora("long_k_many_adapters", FL, HF, 65, 1, 16259, 300, 40, given=True, pad=3)],
                         ids=lambda p: p.name)
def test_rows_sorted_over_many_adapters(lib, p):
    print(f"[case] {p.name}", flush=True)
    d = inputs(p)
    call = Call(lib, p, d)
    got = call.result(nan=True)
    kernels = lib.last_dispatch().kernels()
    assert kernels[0].startswith("map") and set(SORTED) <= set(kernels)
    same_bits(got, documented(p, d, base_bits(p, d)))


@pytest.mark.parametrize("m,n,k,adapters,rank,sorts", [
    (200, 128, 512, 2048, 64, False), (200, 128, 512, 256, 64, False), (800, 128, 512, 2048, 16, False),
    (100, 1024, 1024, 2048, 256, False), (400, 3000, 200, 256, 64, True), (400, 3000, 200, 32, 64, True),
    (1600, 4096, 4096, 32, 4, True), (1600, 4096, 4096, 256, 64, True), (8120, 64, 112, 20, 2, True),
    (2229, 539, 64, 4, 9, True)])
def test_rows_are_sorted_only_where_that_is_faster(lib, m, n, k, adapters, rank, sorts):
    """A slot per adapter costs more than it saves a few rows of many adapters
    (up to seven times the time); many rows and long ones gain up to half."""
    g = torch.Generator(device="cuda").manual_seed(m)
    rnd = lambda *z: torch.randn(*z, generator=g, device="cuda")
    x, base = rnd(m, k), rnd(m, n)
    a, b = (rnd(adapters, rank, k) * k ** -0.5).bfloat16(), rnd(adapters, n, rank).bfloat16()
    ids = torch.randint(0, adapters, (m,), generator=g, device="cuda").int()
    shape = B.make_lora_shape(BF, BF, m, n, k, adapters, rank)
    scratch = torch.empty(lib.lora_linear_scratch_bytes(shape), dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, device="cuda")
    lib.lora_linear(shape, None, base, a, b, None, None, x, ids, out, scratch)
    assert lib.last_dispatch().kernels()[0].startswith("map") == sorts


def test_sorted_rows_at_the_adapters_ends(lib):
    """First and last adapter, adapters whose rows end at, before and behind a
    tile's 16, ids without an adapter and bad ids beside them."""
    p = Lora("ends", BF, BF, 1300, 480, 1000, 150, 16, given=True, none=0.0)
    d = inputs(p)
    ids = d["ids"]
    ids[:] = 149
    at = 0
    for a, rows in ((0, 16), (63, 15), (64, 17), (65, 1), (127, 32), (128, 33), (0xFFFFFFFF, 31), (150, 2), (0x7FFFFFFF, 1)):
        ids[at: at + rows] = a
        at += rows
    ids[:] = np.random.default_rng(3).permutation(ids)
    call = Call(lib, p, d)
    got = call.result(nan=True)
    assert lib.last_dispatch().kernels()[0].startswith("map")
    same_bits(got, documented(p, d, base_bits(p, d)))


@pytest.mark.parametrize("p", [Lora("staged_to_the_end", BF, BF, 3, 40, 16256, 4, 8, none=0.0),
                               Lora("staged_four", HF, HF, 4, 40, 3984, 4, 8, none=0.0),
                               Lora("staged_one", FL, FL, 1, 40, 16256, 4, 8, none=0.0),
                               Lora("beyond", BF, BF, 3, 40, 16257, 4, 8, none=0.0),
                               Lora("given_one", FL, BF, 1, 300, 520, 6, 16, given=True, none=0.0),
                               Lora("given_few", FL, HF, 33, 131, 77, 6, 12, given=True)], ids=lambda p: p.name)
def test_rows_at_the_staging_limit(lib, p):
    print(f"[case] {p.name}", flush=True)
    d = inputs(p)
    call = Call(lib, p, d)
    got = call.result()
    assert lib.last_dispatch().kernels()[0].startswith("map") == (p.k > 16256)
    same_bits(got, documented(p, d, base_bits(p, d)))


@pytest.mark.parametrize("ps", [(Lora("many", BF, BF, 1500, 700, 628, 130, 16), Lora("chunk", BF, BF, 1300, 1024, 264, 6, 16, runs=4)),
                                (Lora("wide", BF, BF, 2, 32768, 136, 8, 16), Lora("few", BF, FL, 9, 256, 136, 8, 16))],
                         ids=["sorted", "rows"])
def test_two_graphs_that_share_a_scratch(lib, ps):
    """Replayed in turn on new rows and adapters, with eager work between."""
    calls = [Call(lib, p, inputs(p)) for p in ps]
    scratch = max((c.scratch for c in calls), key=lambda t: t.numel())
    graphs = []
    for call in calls:
        call.scratch = scratch
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    g = torch.Generator().manual_seed(6)
    for rep in range(5):
        want = []
        for call in calls:
            p = call.p
            call.x.copy_(torch.randn(p.m, p.k, generator=g))
            call.ids.copy_(torch.randint(-1, p.n_adapters, (p.m,), generator=g).int())
            call()
            torch.cuda.synchronize()
            want.append(call.out.clone())
            call.out[: p.m * p.n].zero_()
        scratch.fill_(rep * 41)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for call, w in zip(calls, want):
            assert torch.equal(call.out.view(torch.int32), w.view(torch.int32)), rep
