"""The few-token expert FFN (eidm_moe_ffn_decode) in each of its forms on the
GPU, the form asserted by the dispatch receipt: each token by itself at the
limits of its rows and experts, and tokens that share the experts' reads."""
import numpy as np
import pytest
import torch

import oracle
from expert_id_matmul_amd import binding as B
from expert_id_matmul_amd import workloads as W
from helpers import assert_close
from test_gpu_moe_decode import Call, F, check_bits, shape_of

pytestmark = pytest.mark.gpu

BF, HF, FL = W.DT_BF16, W.DT_F16, W.DT_F32
TORCH = {FL: torch.float32, HF: torch.float16, BF: torch.bfloat16}


def problem(lib, fw, bias=True, renorm=True, pad=0):
    """A call on inputs made on the device (`pad` NaN scalars after each expert)."""
    g = torch.Generator(device="cuda").manual_seed(fw.seed)
    w = []
    for rows, cols in ((fw.inter, fw.hidden), (fw.inter, fw.hidden), (fw.hidden, fw.inter)):
        t = torch.full((fw.n_experts, rows * cols + pad), float("nan"), dtype=TORCH[fw.dtype], device="cuda")
        for e in range(fw.n_experts):
            t[e, : rows * cols] = torch.randn(rows * cols, generator=g, device="cuda") * cols ** -0.5
        w.append(t)
    x = torch.randn(fw.m, fw.hidden, generator=g, device="cuda")
    logits = torch.randn(fw.m, fw.n_experts, generator=g, device="cuda")
    b = torch.rand(fw.n_experts, generator=g, device="cuda") * 0.2 - 0.1 if bias else None
    return Call(lib, fw, shape_of(fw, pad), w, x, logits, b, renorm)


EACH = ["decode_gate_up_one", "decode_down_one"]
SHARED_COMBINED = ["decode_gate_up", "decode_down_combine"]  # all rows of h beside each other in LDS
SHARED = ["decode_gate_up", "decode_down", "combine"]


def form_of(lib):
    return [k for k in lib.last_dispatch().kernels() if k != "route"]


def check_form(lib, call, form, route=None):
    """The call's kernels; route: whether routing is a launch of its own."""
    call()
    assert form_of(lib) == form
    if route is not None:
        assert ("route" in lib.last_dispatch().kernels()) == route


def check_oracle(call):
    fw = call.fw
    raw = [t.view(torch.uint8).cpu().numpy().reshape(-1) for t in call.w]
    bias = None if call.bias is None else call.bias.cpu().numpy()
    ids, gates, _, _ = oracle.route(call.logits.cpu().numpy(), bias, fw.top_k, renormalize=call.renorm)
    got = call.ids.cpu().numpy().view(np.uint32)
    assert np.array_equal(got, ids.reshape(-1))
    want, _ = oracle.moe_ffn(fw.dtype, fw.m, fw.hidden, fw.inter, fw.top_k, fw.n_experts,
                             call.shape.gate_up_stride_bytes, call.shape.down_stride_bytes, *raw,
                             call.x.cpu().numpy(), ids, gates)
    assert_close(call.out.cpu().numpy()[: want.size].reshape(want.shape), want, what=fw.name)


@pytest.mark.parametrize("fw", [F("rows_beside_many_experts", BF, 1, 12288, 24, 2, 300, 81, 0.05),
                                F("wide_top_k_beside_many_experts", HF, 1, 16384, 8, 12, 300, 82, 0.05),
                                F("longest_rows_most_experts", BF, 1, 32768, 4, 3, 2048, 83, 0.05),
                                F("longest_rows_f32", FL, 1, 32768, 12, 2, 4, 84, 0.05),
                                F("longest_inner_rows", BF, 1, 40, 32768, 1, 3, 85, 0.05),
                                F("longest_inner_rows_two_slots", HF, 1, 40, 32768, 2, 3, 86, 0.05)],
                         ids=lambda f: f.name)
def test_longest_rows(lib, fw):
    """Rows up to the limit, staged in LDS beside the router's scores."""
    print(f"[case] {fw.name}", flush=True)
    call = problem(lib, fw)
    check_form(lib, call, SHARED if fw.inter == 32768 and fw.top_k > 1 else EACH, route=False)  # h beyond LDS
    check_bits(lib, call)
    check_oracle(call)


@pytest.mark.parametrize("m,hidden,inter,top_k,experts,form", [
    (2, 2048, 768, 8, 128, EACH), (16, 256, 128, 8, 128, EACH), (16, 256, 128, 8, 2048, EACH),
    (64, 256, 128, 8, 128, SHARED), (24, 336, 216, 8, 512, SHARED), (8, 2048, 768, 8, 128, SHARED)])
def test_the_faster_form_is_taken(lib, m, hidden, inter, top_k, experts, form):
    """Tokens by themselves where sharing would cost more than it saves
    (measured 1.3 to 1.7 times the time), together where not (1.1 to 2.5)."""
    call = problem(lib, F("rule", BF, m, hidden, inter, top_k, experts, 104, 0.05))
    call()
    assert form_of(lib)[0] == form[0]
    check_bits(lib, call)


# shape, form, routing launch
SHARING = [(F("odd_f32", FL, 13, 1001, 363, 5, 37, 91, 0.05), SHARED_COMBINED, True),
           (F("routed_in_the_block", BF, 5, 2048, 768, 8, 16, 92, 0.05), SHARED_COMBINED, False),
           (F("odd_f16", HF, 6, 1101, 701, 6, 8, 93, 0.05), SHARED_COMBINED, False),
           (F("odd_f32_few", FL, 4, 901, 1303, 3, 4, 94, 0.05), SHARED_COMBINED, False),
           (F("f32_rows_beyond_lds", FL, 8, 1003, 901, 4, 4, 95, 0.05), SHARED, False),
           (F("hidden_below_a_granule", BF, 64, 7, 32768, 4, 8, 96, 0.05), SHARED, True),
           (F("inter_below_a_granule", FL, 64, 32768, 5, 4, 8, 97, 0.05), SHARED, True),
           (F("inter_below_a_granule_combined", HF, 48, 32768, 3, 4, 6, 98, 0.05), SHARED_COMBINED, True),
           (F("experts_in_passes", BF, 20, 4096, 1024, 2, 3, 99, 0.05), SHARED, True),
           (F("most_slots", BF, 64, 512, 320, 16, 512, 100, 0.05), SHARED, True),
           (F("most_experts", HF, 64, 512, 256, 16, 2048, 101, 0.05), SHARED, True),
           (F("routed_beside_300_experts", BF, 8, 2048, 768, 16, 300, 102, 0.05), SHARED, True),
           (F("slots_beyond_lds", BF, 1, 256, 20000, 8, 12, 103, 0.05), SHARED, False)]


@pytest.mark.parametrize("pad", [0, 3], ids=["dense", "padded"])
@pytest.mark.parametrize("fw,form,route", SHARING, ids=lambda v: getattr(v, "name", ""))
def test_tokens_that_share_experts(lib, fw, form, route, pad):
    print(f"[case] {fw.name} pad {pad}", flush=True)
    call = problem(lib, fw, bias=pad == 0, renorm=pad == 0, pad=pad)
    check_form(lib, call, form, route)
    check_bits(lib, call)
    if fw.hidden * fw.inter * fw.m * fw.top_k <= 7e7:  # the oracle's time
        check_oracle(call)


@pytest.mark.parametrize("m", [2, 3, 4, 5, 8, 9, 16, 17, 33, 64])
def test_shared_reads_give_each_token_its_own_bits(lib, m):
    """Eight experts of uneven popularity read together, up to 64 rows of one;
    a token alone has the same bits."""
    print(f"[case] batch {m}", flush=True)
    fw = F("batch", BF, m, 4096, 2048, 4, 8, 111, 0.05)
    call = problem(lib, fw, bias=False)
    call.logits += 2 * torch.randn(8, generator=torch.Generator().manual_seed(m)).cuda()
    check_form(lib, call, SHARED_COMBINED if m <= 4 else SHARED)
    check_bits(lib, call)
    t = m - 1
    one = F("one", BF, 1, 4096, 2048, 4, 8, 111, 0.05)
    alone = Call(lib, one, shape_of(one), call.w, call.x[t:].contiguous(), call.logits[t:].contiguous(), None)
    check_form(lib, alone, EACH)
    torch.cuda.synchronize()
    assert torch.equal(alone.out[:4096].view(torch.int32), call.out[t * 4096: m * 4096].view(torch.int32))


@pytest.mark.parametrize("dtype", [HF, BF, FL], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,form", [(6, SHARED_COMBINED), (20, SHARED)], ids=["combined", "rows"])
def test_shared_reads_at_the_scalar_alignment(lib, m, form, dtype):
    """Weights one scalar and activations four bytes past a 16-byte boundary."""
    fw = F("unaligned", dtype, m, 1101, 701, 6, 8, 112, 0.05)
    call = problem(lib, fw)
    size = W.DTYPE_SIZE[dtype]

    def shifted(t, by):
        raw = t.contiguous().view(torch.uint8).reshape(-1)
        buf = torch.empty(raw.numel() + 16, dtype=torch.uint8, device="cuda")
        buf[by: by + raw.numel()] = raw
        return buf[by: by + raw.numel()]

    call.w = [shifted(t, size) for t in call.w]
    call.x = shifted(call.x, 4).view(torch.float32)
    check_form(lib, call, form)
    check_bits(lib, call)


@pytest.mark.parametrize("m,form", [(9, SHARED_COMBINED), (24, SHARED)], ids=["combined", "rows"])
def test_non_finite_tokens_beside_others_in_a_tile(lib, m, form):
    fw = F("specials", BF, m, 2048, 768, 4, 6, 113, 0.05)
    call = problem(lib, fw)
    call.x[1, 5], call.x[3, 2047], call.x[4, 0] = float("inf"), float("nan"), -float("inf")
    call.x[6] = 1e-42  # subnormal
    check_form(lib, call, form)
    check_bits(lib, call, nan=True)
    out = call.out[: m * 2048].view(m, 2048)
    sound = [t for t in range(m) if t not in (1, 3, 4)]
    assert torch.isfinite(out[sound]).all()


@pytest.mark.parametrize("m,form", [(9, SHARED_COMBINED), (24, SHARED)], ids=["combined", "rows"])
def test_unpicked_experts_are_not_read_into_shared_results(lib, m, form):
    fw = F("unpicked", HF, m, 2048, 768, 4, 8, 114, 0.05)
    call = problem(lib, fw, bias=False)
    call.logits[:, 6:] = -30.0
    check_form(lib, call, form)
    torch.cuda.synchronize()
    before = call.out.clone()
    assert max(call.ids.tolist()) < 6
    for t in call.w:
        t[6:] = float("nan")
    call()
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int32), call.out.view(torch.int32))


@pytest.mark.parametrize("dtype,m,form", [(BF, 5, SHARED_COMBINED), (FL, 9, SHARED_COMBINED), (HF, 24, SHARED)],
                         ids=["routed_in_the_block", "combined", "rows"])
def test_graphs_of_shared_reads_replay_to_the_eager_bits(lib, dtype, m, form):
    """Two captured calls that share a scratch, replayed in turn on new
    inputs with eager work between."""
    fw = F("graph", dtype, m, 2048, 400, 6, 8, 115, 0.05)
    calls = [problem(lib, fw), problem(lib, fw)]
    calls[1].scratch = calls[0].scratch
    calls[1].w = calls[0].w
    for call in calls:
        check_form(lib, call, form)
    torch.cuda.synchronize()
    graphs = []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    g = torch.Generator().manual_seed(m)
    for rep in range(5):
        want = []
        for call in calls:
            call.x.copy_(torch.randn(call.x.shape, generator=g))
            call.logits.copy_(torch.randn(call.logits.shape, generator=g))
            call()
            torch.cuda.synchronize()
            want.append(call.out.clone())
            call.out[: fw.m * fw.hidden].zero_()
        calls[0].scratch.fill_(rep * 37)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for call, w in zip(calls, want):
            assert torch.equal(call.out.view(torch.int32), w.view(torch.int32)), rep


@pytest.mark.parametrize("m,form", [(9, SHARED_COMBINED), (24, SHARED)], ids=["combined", "rows"])
def test_shared_reads_on_two_streams_at_once(lib, m, form):
    calls, want = [], []
    for i in range(2):
        call = problem(lib, F("streams", BF, m, 2048, 768, 4, 6, 116 + i, 0.05))
        check_form(lib, call, form)
        torch.cuda.synchronize()
        want.append(call.out.clone())
        call.out[: m * 2048].zero_()
        calls.append(call)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, call in zip(streams, calls):
            call(stream=s)
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        assert torch.equal(call.out.view(torch.int32), w.view(torch.int32))
