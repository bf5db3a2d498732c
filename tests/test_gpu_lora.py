"""Low-rank adapters beside a shared projection (eidm_lora_linear) on the GPU:
the documented order bit for bit, the oracle within the derived bound."""
import numpy as np
import pytest
import torch

import oracle
from expert_id_matmul_amd import binding as B
from expert_id_matmul_amd import workloads as W
from helpers import assert_close, check_guarded, ids_to_dev, poisoned_output, to_dev
from lora_cases import NO_ADAPTER, Lora, base_bits, bound, documented, inputs

pytestmark = pytest.mark.gpu

BF, HF, FL = W.DT_BF16, W.DT_F16, W.DT_F32
CASES = [Lora("one_row", BF, BF, 1, 128, 256, 4, 16),
         Lora("unit_sizes", FL, FL, 1, 1, 1, 1, 1, ranks=False, none=0.0),
         Lora("below_a_granule", HF, BF, 3, 5, 7, 2, 3),
         Lora("odd", HF, FL, 9, 111, 203, 8, 11, pad=3),
         Lora("odd_bf16", BF, BF, 33, 77, 331, 5, 13, pad=1),
         Lora("rank_above_a_round", BF, BF, 6, 96, 192, 3, 200),
         Lora("most_ranks", HF, HF, 18, 130, 150, 3, 256, ranks=False),
         Lora("each_its_own", BF, BF, 40, 200, 384, 64, 24),
         Lora("batch_of_64", BF, HF, 64, 272, 520, 9, 16),
         Lora("batch_of_65", BF, BF, 65, 272, 520, 9, 16),
         Lora("most_adapters", FL, BF, 50, 40, 64, 2048, 4),
         Lora("prompts", BF, BF, 700, 192, 320, 6, 16, runs=9),
         Lora("prompts_odd", HF, HF, 333, 117, 221, 5, 10, runs=7, pad=1),
         Lora("prompts_f32", FL, FL, 260, 96, 160, 4, 33, runs=5, scales=False, ranks=False),
         Lora("one_prompt", BF, BF, 1100, 160, 256, 3, 64, runs=1, none=0.0),
         Lora("scattered", BF, BF, 900, 96, 128, 40, 8),
         Lora("nobody", BF, BF, 20, 64, 64, 3, 8, none=1.0),
         Lora("given", BF, BF, 12, 130, 96, 4, 16, given=True),
         Lora("given_odd", FL, HF, 77, 63, 45, 6, 19, given=True, pad=5),
         Lora("given_prompts", FL, BF, 2100, 264, 136, 7, 16, runs=23, given=True),
         Lora("given_f32", FL, FL, 130, 100, 70, 5, 40, runs=6, given=True),
         Lora("long_rows", BF, BF, 5, 72, 8200, 3, 8),
         Lora("one_row_beyond_lds", BF, BF, 1, 24, 20003, 3, 8, none=0.0),
         Lora("rows_beyond_lds", HF, FL, 7, 40, 17000, 3, 20),
         Lora("prompts_many_ranks_f32", FL, FL, 1500, 48, 100, 3, 40, runs=5),
         Lora("prompts_many_ranks", BF, HF, 1450, 40, 203, 4, 57, runs=8, given=True)]


def shape_of(p):
    return B.make_lora_shape(p.w_dtype, p.a_dtype, p.m, p.n, p.k, p.n_adapters, p.max_rank, p.arith, p.a_stride,
                             p.b_stride)


class Call:
    def __init__(self, lib, p, d):
        self.lib, self.p, self.shape = lib, p, shape_of(p)
        dev = lambda z: None if z is None else to_dev(z)
        self.w, self.base, self.a, self.b = dev(d["w"]), dev(d["base"]), to_dev(d["a"]), to_dev(d["b"])
        self.ranks = None if d["ranks"] is None else ids_to_dev(d["ranks"])
        self.scales, self.x, self.ids = dev(d["scales"]), to_dev(d["x"]), ids_to_dev(d["ids"])
        self.out = poisoned_output(p.m * p.n)
        self.scratch = torch.full((lib.lora_linear_scratch_bytes(self.shape),), 0xFF, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        self.lib.lora_linear(self.shape, self.w, self.base, self.a, self.b, self.ranks, self.scales, self.x, self.ids,
                             self.out, self.scratch, stream=stream)

    def result(self, nan=False):
        self()
        torch.cuda.synchronize()
        return check_guarded(self.out, self.p.m * self.p.n, nan).reshape(self.p.m, self.p.n)


def run_oracle(p, d):
    return oracle.lora_linear(p.w_dtype, p.a_dtype, p.m, p.n, p.k, p.n_adapters, p.max_rank, p.a_stride, p.b_stride,
                              d["w"], d["base"], d["a"], d["b"], d["ranks"], d["scales"], d["x"], d["ids"])


def same_bits(got, want):
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    live = ~np.isnan(want)
    np.testing.assert_array_equal(got[live].view(np.uint32), want[live].view(np.uint32))


@pytest.mark.parametrize("p", CASES, ids=lambda p: p.name)
def test_documented_bits_and_the_oracle(lib, p):
    print(f"[case] {p.name}", flush=True)
    d = inputs(p)
    got = Call(lib, p, d).result()
    same_bits(got, documented(p, d, base_bits(p, d)))
    err = np.abs(got.astype(np.float64) - run_oracle(p, d))
    assert (err <= bound(p, d)).all(), float((err / bound(p, d)).max())


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 47, 64, 65, 96, 128, 129, 257])
def test_every_batch_size(lib, m):
    """Rows around every tile size; a row's bits do not depend on the batch."""
    print(f"[case] batch {m}", flush=True)
    p = Lora("batch", BF, BF, m, 136, 264, 5, 16, seed=m)
    d = inputs(p)
    call = Call(lib, p, d)
    got = call.result()
    same_bits(got, documented(p, d, base_bits(p, d)))
    t = m - 1
    one = Lora("alone", BF, BF, 1, 136, 264, 5, 16)
    alone = Call(lib, one, dict(d, x=d["x"][t:], ids=d["ids"][t:])).result()
    same_bits(alone[0], got[t])


@pytest.mark.parametrize("dtype,m,n,k", [(BF, 500, 750, 136), (HF, 512, 768, 131), (FL, 481, 737, 200), (BF, 97, 2000, 264),
                                         (HF, 130, 1500, 72), (FL, 60, 1530, 140)], ids=lambda v: str(v))
def test_projection_tiles_of_every_size(lib, dtype, m, n, k):
    """16 x 16 to 32 x 48 outputs a block, whole and cut: the bits of
    eidm_matmul_id's Direct route."""
    g = torch.Generator(device="cuda").manual_seed(m)
    tdt = {HF: torch.float16, BF: torch.bfloat16, FL: torch.float32}[dtype]
    x = torch.randn(m, k, generator=g, device="cuda")
    w = (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(tdt)
    a, b = torch.zeros(1, 4, k, device="cuda", dtype=tdt), torch.zeros(1, n, 4, device="cuda", dtype=tdt)
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    shape = B.make_lora_shape(dtype, dtype, m, n, k, 1, 4)
    scratch = torch.full((lib.lora_linear_scratch_bytes(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    out = poisoned_output(m * n)
    lib.lora_linear(shape, w, None, a, b, None, None, x, ids, out, scratch)
    assert "lora_base" in lib.last_dispatch().kernels()
    want = torch.empty(m, n, device="cuda")
    s = B.make_shape(dtype, m, n, k, 1, 1, n * k * W.DTYPE_SIZE[dtype])
    lib.matmul_id(s, B.DIRECT, w, x, torch.zeros(m, 1, dtype=torch.int32, device="cuda"), want)
    torch.cuda.synchronize()
    check_guarded(out, m * n)
    assert torch.equal(out[: m * n].view(m, n).view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("p", [Lora("split_bf16", BF, BF, 40, 128, 256, 6, 16, arith=1),
                               Lora("split_one", BF, BF, 1, 272, 520, 4, 8, arith=1),
                               Lora("split_f16", HF, HF, 300, 144, 264, 5, 24, runs=4, arith=1),
                               Lora("split_17", BF, FL, 17, 48, 1000, 3, 5, arith=1),
                               Lora("split_64", HF, BF, 64, 208, 136, 7, 16, arith=1),
                               Lora("split_prompts", BF, BF, 600, 160, 392, 6, 16, runs=5, arith=1)],
                         ids=lambda p: p.name)
def test_split16_projection(lib, p):
    """The shared projection in the split-16 arithmetic has eidm_matmul_id's
    bits there; the adapters are added in the documented order."""
    print(f"[case] {p.name}", flush=True)
    d = inputs(p)
    call = Call(lib, p, d)
    got = call.result()
    s = B.make_shape(p.w_dtype, p.m, p.n, p.k, 1, 1, p.n * p.k * 2, arith=B.ARITH_SPLIT16)
    base = torch.empty(p.m, p.n, device="cuda")
    scratch = torch.empty(lib.query(s, B.DIRECT).scratch_bytes, dtype=torch.uint8, device="cuda")
    lib.matmul_id(s, B.DIRECT, call.w, call.x, torch.zeros(p.m, 1, dtype=torch.int32, device="cuda"), base, scratch)
    same_bits(got, documented(p, d, base.cpu().numpy()))
    assert_close(got, run_oracle(p, d), what=p.name)


@pytest.mark.parametrize("dtype,m,n,k", [(BF, 1300, 1500, 136), (HF, 1030, 2051, 264), (BF, 2048, 1024, 8),
                                         (HF, 4100, 515, 1000), (BF, 130, 8200, 392), (BF, 16384, 129, 128)],
                         ids=lambda v: str(v))
def test_split16_projection_of_many_rows(lib, dtype, m, n, k):
    """Sizes that fill the device with 128 x 128 tiles: every output's bits
    against eidm_matmul_id's Direct route, with adapters on some rows."""
    print(f"[case] {dtype} {m} {n} {k}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(k)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    tdt = torch.float16 if dtype == HF else torch.bfloat16
    x, w = rnd(m, k), (rnd(n, k) * k ** -0.5).to(tdt)
    a, b = rnd(2, 4, k).to(tdt), rnd(2, n, 4).to(tdt)
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    ids[m // 2: m // 2 + 3] = 1
    shape = B.make_lora_shape(dtype, dtype, m, n, k, 2, 4, arith=B.ARITH_SPLIT16)
    scratch = torch.full((lib.lora_linear_scratch_bytes(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    out = poisoned_output(m * n)
    lib.lora_linear(shape, w, None, a, b, None, None, x, ids, out, scratch)
    torch.cuda.synchronize()
    assert "dense_split16" in lib.last_dispatch().kernels()
    s = B.make_shape(dtype, m, n, k, 1, 1, n * k * 2, arith=B.ARITH_SPLIT16)
    base, ds = torch.empty(m, n, device="cuda"), torch.empty(lib.query(s, B.DIRECT).scratch_bytes, dtype=torch.uint8, device="cuda")
    lib.matmul_id(s, B.DIRECT, w, x, torch.zeros(m, 1, dtype=torch.int32, device="cuda"), base, ds)
    torch.cuda.synchronize()
    got = out[: m * n].view(m, n)
    plain = ids < 0
    assert torch.equal(got[plain].view(torch.int32), base[plain].view(torch.int32))
    check_guarded(out, m * n)
    low = (x[~plain].double() @ a[1].double().t()) @ b[1].double().t()
    err = (got[~plain].double() - base[~plain].double() - low).abs().max() / low.abs().max()
    assert err < 2e-5


@pytest.mark.parametrize("dtype", [HF, BF], ids=["f16", "bf16"])
def test_split16_projection_of_many_rows_with_special_values(lib, dtype):
    """Infinite, NaN, subnormal and (for f16) out-of-range activations: the
    same values as eidm_matmul_id's Direct route, and other rows untouched."""
    m, n, k = 1100, 1920, 72
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(m, k, generator=g, device="cuda")
    tdt = torch.float16 if dtype == HF else torch.bfloat16
    w = (torch.randn(n, k, generator=g, device="cuda") * 0.1).to(tdt)
    clean = x.clone()
    x[3, 5], x[130, 71], x[131, 0], x[1099, 8] = float("inf"), float("nan"), -float("inf"), 1e6
    x[700], x[701, 3] = 1e-42, 3.4e38
    odd = [3, 130, 131, 700, 701, 1099]
    a, b = torch.zeros(1, 2, k, device="cuda", dtype=tdt), torch.zeros(1, n, 2, device="cuda", dtype=tdt)
    ids = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    shape = B.make_lora_shape(dtype, dtype, m, n, k, 1, 2, arith=B.ARITH_SPLIT16)
    scratch = torch.full((lib.lora_linear_scratch_bytes(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    out, plain = (torch.empty(m, n, device="cuda") for _ in range(2))
    lib.lora_linear(shape, w, None, a, b, None, None, x, ids, out, scratch)
    assert "dense_split16" in lib.last_dispatch().kernels()
    lib.lora_linear(shape, w, None, a, b, None, None, clean, ids, plain, scratch)
    s = B.make_shape(dtype, m, n, k, 1, 1, n * k * 2, arith=B.ARITH_SPLIT16)
    want, ds = torch.empty(m, n, device="cuda"), torch.empty(lib.query(s, B.DIRECT).scratch_bytes, dtype=torch.uint8, device="cuda")
    lib.matmul_id(s, B.DIRECT, w, x, torch.zeros(m, 1, dtype=torch.int32, device="cuda"), want, ds)
    torch.cuda.synchronize()
    nan = want.isnan()
    assert nan.any() and torch.equal(nan, out.isnan())
    assert torch.equal(out[~nan].view(torch.int32), want[~nan].view(torch.int32))
    same = torch.ones(m, dtype=torch.bool, device="cuda")
    same[odd] = False
    assert torch.equal(out[same].view(torch.int32), plain[same].view(torch.int32))


@pytest.mark.parametrize("given", [False, True], ids=["weights", "given"])
@pytest.mark.parametrize("m", [7, 70, 300])
def test_bad_ids_rank_zero_and_rows_without_an_adapter(lib, m, given):
    p = Lora("edges", BF, BF, m, 72, 136, 6, 12, given=given, none=0.3, runs=0)
    d = inputs(p)
    d["ids"][[0, m // 2]] = [p.n_adapters, 0x7FFFFFFF]
    d["ids"][[1, m - 1]] = NO_ADAPTER
    d["ids"][2] = 4
    d["ranks"][4] = 0
    got = Call(lib, p, d).result(nan=True)
    base = base_bits(p, d)
    same_bits(got, documented(p, d, base))
    assert np.isnan(got[[0, m // 2]]).all() and np.isfinite(np.delete(got, [0, m // 2], 0)).all()
    same_bits(got[[1, m - 1, 2]], base[[1, m - 1, 2]])


def test_elements_past_the_rank_are_not_used(lib):
    p = Lora("past_rank", BF, BF, 20, 64, 96, 4, 24, none=0.0)
    d = inputs(p)
    d["ranks"] = np.array([3, 8, 17, 24], np.uint32)
    want = documented(p, d, base_bits(p, d))
    a = torch.from_numpy(d["a"]).view(torch.bfloat16).view(4, 24, 96)
    b = torch.from_numpy(d["b"]).view(torch.bfloat16).view(4, 64, 24)
    for i, r in enumerate(d["ranks"]):
        a[i, r:] = float("nan")
        b[i, :, r:] = float("inf")
    same_bits(Call(lib, p, d).result(), want)


def test_special_values_stay_in_their_rows_and_adapters(lib):
    """Infinite and NaN activations, adapters, scales and base values."""
    p = Lora("specials", FL, BF, 24, 40, 72, 6, 10, given=True, none=0.1)
    d = inputs(p)
    d["ids"][:8] = [0, 1, 2, 3, 4, 5, NO_ADAPTER, 0]
    d["ranks"][:] = 10
    d["x"][1, 3], d["x"][2, 70], d["x"][6, 0] = np.nan, np.inf, np.nan
    d["base"][0, 5], d["base"][6, 7], d["base"][7] = np.inf, -0.0, 1e-42
    d["scales"][3:6] = [np.inf, 0.0, np.nan]
    got = Call(lib, p, d).result(nan=True)
    same_bits(got, documented(p, d, d["base"]))
    assert got[6, 7] == 0 and np.signbit(got[6, 7])


def test_in_place_on_the_base(lib):
    p = Lora("in_place", FL, HF, 100, 150, 60, 5, 12, runs=7, given=True)
    d = inputs(p)
    call = Call(lib, p, d)
    want = documented(p, d, d["base"])
    call.base = call.out
    call.out[: p.m * p.n].copy_(to_dev(d["base"]).reshape(-1))
    same_bits(call.result(), want)


@pytest.mark.parametrize("dtype", [HF, BF, FL], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("m", [5, 90])
def test_buffers_at_the_scalar_alignment(lib, m, dtype):
    p = Lora("unaligned", dtype, dtype, m, 75, 139, 4, 9, runs=0)
    d = inputs(p)
    call = Call(lib, p, d)
    size = W.DTYPE_SIZE[dtype]

    def shifted(t, by):
        raw = t.contiguous().view(torch.uint8).reshape(-1)
        buf = torch.empty(raw.numel() + 16, dtype=torch.uint8, device="cuda")
        buf[by: by + raw.numel()] = raw
        return buf[by: by + raw.numel()]

    call.w, call.a, call.b = (shifted(t, size) for t in (call.w, call.a, call.b))
    call.x = shifted(call.x, 4).view(torch.float32)
    call.out = poisoned_output(p.m * p.n + 1)[1:]
    same_bits(call.result(), documented(p, d, base_bits(p, d)))


@pytest.mark.parametrize("p", [Lora("graph_few", BF, BF, 8, 256, 512, 8, 16),
                               Lora("graph_one", BF, BF, 1, 256, 512, 8, 16, none=0.0),
                               Lora("graph_prompts", BF, BF, 400, 256, 512, 8, 16, runs=5),
                               Lora("graph_split", BF, BF, 200, 256, 512, 8, 16, runs=5, arith=1),
                               Lora("graph_dense_split", BF, BF, 1024, 2048, 136, 8, 16, runs=5, arith=1),
                               Lora("graph_given", BF, BF, 300, 256, 512, 8, 16, given=True)], ids=lambda p: p.name)
def test_graph_replays_match_eager(lib, p):
    print(f"[case] {p.name}", flush=True)
    call = Call(lib, p, inputs(p))
    call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g = torch.Generator().manual_seed(5)
    for rep in range(5):  # new rows and new adapters each time, with eager calls between the replays
        call.x.copy_(torch.randn(p.m, p.k, generator=g))
        call.ids.copy_(torch.randint(-1, p.n_adapters, (p.m,), generator=g).int())
        call()
        torch.cuda.synchronize()
        eager = call.out.clone()
        call.out[: p.m * p.n].zero_()
        call.scratch.fill_(rep * 41)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out.view(torch.int32), eager.view(torch.int32)), rep


def test_two_streams_at_once(lib):
    calls, want = [], []
    for i, m in enumerate((6, 300)):
        p = Lora("streams", BF, BF, m, 256, 512, 8, 16, seed=i + 1)
        call = Call(lib, p, inputs(p))
        call()
        torch.cuda.synchronize()
        want.append(call.out.clone())
        calls.append(call)
    streams = [torch.cuda.Stream() for _ in calls]
    for call in calls:
        call.out[: call.p.m * call.p.n].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, call in zip(streams, calls):
            call(stream=s)
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        assert torch.equal(call.out.view(torch.int32), w.view(torch.int32))


def test_projection_with_adapters_then_the_expert_layer(lib):
    """A served layer: a shared projection with every request's adapter, its
    rows routed through the few-token expert layer, adapters added to the
    experts' combined rows; each step against the separate operators."""
    m, hid, inter, E, k = 12, 256, 96, 10, 3
    p = Lora("layer", BF, BF, m, hid, hid, 7, 16, seed=3)
    q = Lora("after", BF, BF, m, hid, hid, 7, 8, given=True, seed=4)
    d, d2 = inputs(p), inputs(q)
    g = torch.Generator().manual_seed(9)
    w = [(torch.randn(E, a, b, generator=g) * 0.06).bfloat16().cuda() for a, b in ((inter, hid), (inter, hid), (hid, inter))]
    logits = torch.randn(m, E, generator=g).cuda()
    first, last = Call(lib, p, d), Call(lib, q, d2)
    fs = B.make_ffn_shape(B.BF16, m, hid, inter, k, E)
    ids, gates = torch.empty(m, k, dtype=torch.int32, device="cuda"), torch.empty(m, k, device="cuda")
    rows, mid = torch.empty(m, hid, device="cuda"), torch.empty(m, hid, device="cuda")
    scratch = torch.empty(lib.moe_ffn_decode_scratch_bytes(fs), dtype=torch.uint8, device="cuda")

    first.out, last.x, last.base = rows, rows, mid
    last.out = torch.empty(m, hid, device="cuda")

    def layer():
        first()
        lib.moe_ffn_decode(fs, *w, rows, logits, None, ids, gates, mid, scratch)
        last()

    layer()
    torch.cuda.synchronize()
    want_rows = documented(p, d, base_bits(p, d))
    same_bits(rows.cpu().numpy(), want_rows)
    big = torch.empty(lib.moe_ffn_scratch_bytes(fs), dtype=torch.uint8, device="cuda")
    out = torch.empty(m, hid, device="cuda")
    lib.moe_ffn(fs, B.DIRECT, *w, rows, logits, None, ids, gates, out, big)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int32), mid.view(torch.int32))
    want = documented(q, dict(d2, x=want_rows, base=out.cpu().numpy()), out.cpu().numpy())
    same_bits(last.out.cpu().numpy(), want)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for rep in range(4):
        logits.copy_(torch.randn(m, E, generator=g))
        layer()
        torch.cuda.synchronize()
        eager = last.out.clone()
        last.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.view(torch.int32), last.out.view(torch.int32)), rep


@pytest.mark.parametrize("p", [Lora("full_decode", BF, BF, 32, 1536, 4096, 64, 64),
                               Lora("full_one", BF, BF, 1, 4096, 4096, 16, 16, none=0.0),
                               Lora("full_chunk", BF, BF, 512, 768, 2048, 8, 16, runs=4)], ids=lambda p: p.name)
def test_full_sizes(lib, p):
    print(f"[case] {p.name}", flush=True)
    d = inputs(p)
    same_bits(Call(lib, p, d).result(), documented(p, d, base_bits(p, d)))


def test_rows_past_32_bit_offsets(lib):
    """Rows whose elements lie past 2^31 in the given and the output rows, on
    sampled rows (2^31 elements are 8 GiB)."""
    p = Lora("far", FL, BF, 70000, 32768, 16, 3, 4, given=True, pad=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(p.m, p.k, generator=g, device="cuda")
    a = torch.randn(3, 4, 16, generator=g, device="cuda").bfloat16()
    b = torch.randn(3, p.n, 4, generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, 3, (p.m,), generator=g, device="cuda").int()
    base = torch.empty(p.m, p.n, device="cuda")
    base.copy_(torch.arange(p.m, device="cuda").unsqueeze(1) % 97)
    out = torch.empty(p.m, p.n, device="cuda")
    shape = B.make_lora_shape(B.F32, B.BF16, p.m, p.n, p.k, 3, 4)
    scratch = torch.empty(lib.lora_linear_scratch_bytes(shape), dtype=torch.uint8, device="cuda")
    lib.lora_linear(shape, None, base, a, b, None, None, x, ids, out, scratch)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 65535, 65536, 65537, p.m - 2, p.m - 1])
    s = Lora("far", FL, BF, len(rows), p.n, p.k, 3, 4, given=True)
    raw = lambda t: t.cpu().view(torch.uint8).numpy().reshape(-1)
    d = {"x": x[rows.cuda()].cpu().numpy(), "a": raw(a), "b": raw(b), "b32": b.float().cpu().numpy(), "ranks": None,
         "scales": None, "ids": ids[rows.cuda()].cpu().numpy().view(np.uint32), "w": None}
    same_bits(out[rows.cuda()].cpu().numpy(), documented(s, d, base[rows.cuda()].cpu().numpy()))
    # every other row by its own definition, coarsely: the base and a bounded addition
    has = (ids >= 0).unsqueeze(1)
    assert torch.equal(torch.where(has, base, out), base)


def test_tensors_that_the_binding_refuses(lib):
    p = Lora("refuse", BF, BF, 6, 64, 32, 4, 8)
    d = inputs(p)
    good = Call(lib, p, d)
    good()
    for change in (dict(x=good.x.cpu()), dict(x=good.x.t()), dict(x=good.x.half()), dict(x=good.x[:2]),
                   dict(ids=good.ids.long()), dict(ids=good.ids[:5]), dict(ranks=good.ranks[:3]),
                   dict(scales=good.scales[:3]), dict(out=good.out[:64]), dict(scales=good.scales.double())):
        call = Call(lib, p, d)
        for name, t in change.items():
            setattr(call, name, t)
        with pytest.raises(ValueError):
            call()
    base = torch.zeros(6, 64, device="cuda")
    for change, code in ((dict(base=base), B.E_INVALID), (dict(w=None), B.E_INVALID), (dict(w=good.w[:100]), B.E_SIZE),
                         (dict(a=good.a[:100]), B.E_SIZE), (dict(b=good.b[:100]), B.E_SIZE),
                         (dict(scratch=good.scratch[:256]), B.E_SIZE)):
        call = Call(lib, p, d)
        for name, t in change.items():
            setattr(call, name, t)
        with pytest.raises(B.EidmError) as e:
            call()
        assert e.value.code == code
    torch.cuda.synchronize()
