"""The few-token expert FFN (eidm_moe_ffn_decode) on the GPU: bit for bit
eidm_moe_ffn, within the oracle's bar, and sound at the edges."""
import numpy as np
import pytest
import torch

import oracle
from expert_id_matmul_amd import binding as B
from expert_id_matmul_amd import workloads as W
from helpers import assert_close, check_guarded, poisoned_output, to_dev, u32

pytestmark = pytest.mark.gpu

F = W.FfnWorkload
SHAPES = [F("one_token", W.DT_BF16, 1, 256, 128, 4, 16, 11, 0.05),
          F("one_expert", W.DT_F16, 1, 128, 64, 1, 1, 12, 0.05),
          F("unit_sizes", W.DT_F32, 3, 1, 1, 2, 3, 13, 0.5),
          F("below_a_granule", W.DT_BF16, 2, 7, 5, 2, 4, 14, 0.3),
          F("odd_f16", W.DT_F16, 5, 131, 67, 3, 9, 15, 0.05),
          F("odd_bf16", W.DT_BF16, 13, 1001, 363, 5, 37, 16, 0.03),
          F("odd_f32", W.DT_F32, 6, 333, 129, 4, 10, 17, 0.05),
          F("two_rows", W.DT_BF16, 2, 256, 96, 1, 1, 18, 0.05),
          F("four_rows", W.DT_F16, 4, 256, 96, 1, 1, 19, 0.05),
          F("five_rows", W.DT_BF16, 5, 256, 96, 2, 2, 20, 0.05),
          F("nine_rows", W.DT_F32, 9, 256, 96, 2, 2, 21, 0.05),
          F("seventeen_rows", W.DT_BF16, 17, 256, 96, 3, 3, 22, 0.05),
          F("full_batch_few_experts", W.DT_BF16, 64, 320, 160, 6, 6, 23, 0.05),
          F("full_batch", W.DT_F16, 64, 384, 200, 8, 64, 24, 0.05),
          F("top_16", W.DT_BF16, 64, 128, 64, 16, 300, 25, 0.05),
          F("most_experts", W.DT_BF16, 9, 64, 32, 16, 2048, 26, 0.05),
          F("long_rows", W.DT_BF16, 7, 2880, 1408, 4, 8, 27, 0.02),
          F("wide", W.DT_F16, 3, 4100, 40, 2, 5, 28, 0.02)]


def weights(fw, pad=0, seed=None):
    """Device weights [E][rows][cols], `pad` NaN scalars after each expert."""
    dt = {W.DT_F32: torch.float32, W.DT_F16: torch.float16, W.DT_BF16: torch.bfloat16}[fw.dtype]
    g = torch.Generator().manual_seed(fw.seed if seed is None else seed)
    out = []
    for rows, cols in ((fw.inter, fw.hidden), (fw.inter, fw.hidden), (fw.hidden, fw.inter)):
        w = (torch.randn(fw.n_experts, rows * cols, generator=g) * fw.w_std).to(dt)
        if pad:
            w = torch.cat([w, torch.full((fw.n_experts, pad), float("nan"), dtype=dt)], 1)
        out.append(w.contiguous().cuda())
    return out


def shape_of(fw, pad=0):
    size = W.DTYPE_SIZE[fw.dtype]
    stride = (fw.hidden * fw.inter + pad) * size
    return B.make_ffn_shape(fw.dtype, fw.m, fw.hidden, fw.inter, fw.top_k, fw.n_experts, stride, stride)


class Call:
    def __init__(self, lib, fw, shape, w, x, logits, bias, renorm=True):
        self.lib, self.fw, self.shape, self.w = lib, fw, shape, w
        self.x, self.logits, self.bias, self.renorm = x, logits, bias, renorm
        self.ids = torch.full((fw.m * fw.top_k,), -7, dtype=torch.int32, device="cuda")
        self.gates = poisoned_output(fw.m * fw.top_k)
        self.out = poisoned_output(fw.m * fw.hidden)
        # scratch as a program may hand it over: anything in it
        self.scratch = torch.full((lib.moe_ffn_decode_scratch_bytes(shape),), 0xFF, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        self.lib.moe_ffn_decode(self.shape, *self.w, self.x, self.logits, self.bias, self.ids, self.gates, self.out,
                                self.scratch, renormalize=self.renorm, stream=stream)


def separate(lib, fw, shape, w, x, logits, bias, renorm=True):
    """eidm_moe_ffn on the same inputs (Direct: one row at a time)."""
    ids = torch.empty(fw.m, fw.top_k, dtype=torch.int32, device="cuda")
    gates = torch.empty(fw.m, fw.top_k, device="cuda")
    out = torch.empty(fw.m, fw.hidden, device="cuda")
    scratch = torch.empty(lib.moe_ffn_scratch_bytes(shape), dtype=torch.uint8, device="cuda")
    lib.moe_ffn(shape, B.DIRECT, *w, x, logits, bias, ids, gates, out, scratch, renormalize=renorm)
    torch.cuda.synchronize()
    return ids, gates, out


def check_bits(lib, call, nan=False):
    fw = call.fw
    call()
    torch.cuda.synchronize()
    ids, gates, out = separate(lib, fw, call.shape, call.w, call.x, call.logits, call.bias, call.renorm)
    assert np.array_equal(u32(call.ids), u32(ids).reshape(-1))
    g = check_guarded(call.gates, fw.m * fw.top_k, nan)
    o = check_guarded(call.out, fw.m * fw.hidden, nan)
    want = out.cpu().numpy().reshape(-1)
    np.testing.assert_array_equal(g.view(np.uint32), gates.cpu().numpy().reshape(-1).view(np.uint32))
    if nan:
        live = ~np.isnan(want)
        assert np.array_equal(live, ~np.isnan(o))
        o, want = o[live], want[live]
    np.testing.assert_array_equal(o.view(np.uint32), want.view(np.uint32))


@pytest.mark.parametrize("pad", [0, 3], ids=["dense", "padded"])
@pytest.mark.parametrize("fw", SHAPES, ids=lambda f: f.name)
def test_bits_of_the_separate_steps_and_the_oracle(lib, fw, pad):
    print(f"[case] {fw.name} pad {pad}", flush=True)
    w = weights(fw, pad)
    shape = shape_of(fw, pad)
    xh, lh, bh = W.ffn_inputs(fw)
    call = Call(lib, fw, shape, w, to_dev(xh), to_dev(lh), to_dev(bh) if pad == 0 else None, renorm=pad == 0)
    check_bits(lib, call)
    ids, gates, _, _ = oracle.route(lh, bh if pad == 0 else None, fw.top_k, renormalize=pad == 0)
    assert np.array_equal(u32(call.ids), ids.reshape(-1))
    if fw.hidden * fw.inter * fw.m * fw.top_k > 2e8:
        return  # the oracle's time
    raw = [t.view(torch.uint8).cpu().numpy().reshape(-1) for t in w]
    want, _ = oracle.moe_ffn(fw.dtype, fw.m, fw.hidden, fw.inter, fw.top_k, fw.n_experts, shape.gate_up_stride_bytes,
                             shape.down_stride_bytes, *raw, xh, ids, gates)
    assert_close(call.out.cpu().numpy()[: want.size].reshape(want.shape), want, what=fw.name)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 33, 48, 63, 64])
def test_every_batch_gives_each_token_its_own_bits(lib, m):
    """Tokens that share experts in every way (uneven popularity): a token's
    row is the same bits in a batch of m and alone."""
    print(f"[case] batch {m}", flush=True)
    fw = F("batch", W.DT_BF16, m, 264, 136, 4, 12, 31, 0.05)
    w, shape = weights(fw), shape_of(fw)
    g = torch.Generator().manual_seed(m)
    x = torch.randn(m, fw.hidden, generator=g).cuda()
    logits = (torch.randn(m, 12, generator=g) + 2 * torch.randn(12, generator=g)).cuda()
    call = Call(lib, fw, shape, w, x, logits, None)
    check_bits(lib, call)
    t = m - 1
    one = F("one", W.DT_BF16, 1, 264, 136, 4, 12, 31, 0.05)
    alone = Call(lib, one, shape_of(one), w, x[t:].contiguous(), logits[t:].contiguous(), None)
    alone()
    torch.cuda.synchronize()
    assert torch.equal(alone.out[:264].view(torch.int32), call.out[t * 264: m * 264].view(torch.int32))


@pytest.mark.parametrize("dtype", [W.DT_F16, W.DT_BF16], ids=["f16", "bf16"])
def test_weights_at_the_scalar_alignment(lib, dtype):
    """Weights one scalar past a 16-byte boundary."""
    fw = F("unaligned", dtype, 6, 259, 133, 3, 7, 41, 0.05)
    shape = shape_of(fw)
    w = []
    for t in weights(fw):
        buf = torch.empty(t.nbytes + 16, dtype=torch.uint8, device="cuda")
        buf[2: 2 + t.nbytes] = t.view(torch.uint8).reshape(-1)
        w.append(buf[2: 2 + t.nbytes])
    xh, lh, bh = W.ffn_inputs(fw)
    check_bits(lib, Call(lib, fw, shape, w, to_dev(xh), to_dev(lh), to_dev(bh)))


def test_activations_at_four_byte_alignment(lib):
    fw = F("x_unaligned", W.DT_BF16, 5, 260, 132, 3, 7, 42, 0.05)
    xh, lh, bh = W.ffn_inputs(fw)
    buf = torch.empty(xh.size + 4, device="cuda")
    x = buf[1: 1 + xh.size]
    x.copy_(to_dev(xh).reshape(-1))
    check_bits(lib, Call(lib, fw, shape_of(fw), weights(fw), x, to_dev(lh), to_dev(bh)))


def test_non_finite_activations_stay_in_their_tokens(lib):
    fw = F("specials", W.DT_BF16, 9, 256, 128, 4, 6, 43, 0.05)
    w, shape = weights(fw), shape_of(fw)
    xh, lh, bh = W.ffn_inputs(fw)
    xh = xh.copy()
    xh[1, 5], xh[3, 200], xh[4, 0] = np.inf, np.nan, -np.inf
    xh[6] = 1e-42  # subnormal
    xh[7] *= 1e30
    call = Call(lib, fw, shape, w, to_dev(xh), to_dev(lh), to_dev(bh))
    check_bits(lib, call, nan=True)
    out = call.out[: 9 * 256].view(9, 256)
    assert torch.isfinite(out[[0, 2, 5, 6, 8]]).all()


def test_unpicked_experts_are_not_read_into_results(lib):
    """NaN in every expert that no token picks changes nothing."""
    fw = F("unpicked", W.DT_F16, 3, 128, 96, 2, 24, 44, 0.05)
    w, shape = weights(fw), shape_of(fw)
    xh, lh, bh = W.ffn_inputs(fw)
    call = Call(lib, fw, shape, w, to_dev(xh), to_dev(lh), to_dev(bh))
    call()
    torch.cuda.synchronize()
    before = call.out.clone()
    picked = set(call.ids.tolist())
    for t in w:
        for e in range(24):
            if e not in picked:
                t[e] = float("nan")
    call()
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int32), call.out.view(torch.int32))


@pytest.mark.parametrize("m", [1, 6, 24])
def test_graph_replays_match_eager(lib, m):
    print(f"[case] graph {m}", flush=True)
    fw = F("graph", W.DT_BF16, m, 512, 256, 4, 16, 51, 0.05)
    w, shape = weights(fw), shape_of(fw)
    xh, lh, bh = W.ffn_inputs(fw)
    call = Call(lib, fw, shape, w, to_dev(xh), to_dev(lh), to_dev(bh))
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
    rng = np.random.default_rng(m)
    for rep in range(5):  # new inputs each time, with eager work between the replays
        call.x.copy_(torch.from_numpy(rng.standard_normal(xh.shape, np.float32)))
        call.logits.copy_(torch.from_numpy(rng.standard_normal(lh.shape, np.float32)))
        call.scratch.fill_(rep * 37)
        call.out[: fw.m * fw.hidden].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = call.out.clone()
        ids, gates, out = separate(lib, fw, shape, w, call.x, call.logits, call.bias)
        assert torch.equal(got[: fw.m * fw.hidden].view(torch.int32), out.reshape(-1).view(torch.int32)), rep


def test_two_streams_at_once(lib):
    """Calls on two streams with their own scratch do not disturb each other."""
    fw = F("streams", W.DT_BF16, 8, 512, 256, 4, 16, 52, 0.05)
    w, shape = weights(fw), shape_of(fw)
    calls, want = [], []
    for i in range(2):
        g = torch.Generator().manual_seed(i)
        call = Call(lib, fw, shape, w, torch.randn(8, 512, generator=g).cuda(), torch.randn(8, 16, generator=g).cuda(), None)
        want.append(separate(lib, fw, shape, w, call.x, call.logits, None)[2].reshape(-1))
        calls.append(call)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, call in zip(streams, calls):
            call(stream=s)
    torch.cuda.synchronize()
    for call, out in zip(calls, want):
        assert torch.equal(call.out[: out.numel()].view(torch.int32), out.view(torch.int32))


def test_full_size_decode_batches(lib):
    """The benchmark FFN's experts (128 of 768 x 2048, top 8) at 1, 8 and 64
    tokens: every output's bits against the separate steps'."""
    for m in (1, 8, 64):
        print(f"[case] full size, {m} tokens", flush=True)
        fw = F("full", W.DT_BF16, m, 2048, 768, 8, 128, 61, 0.02)
        g = torch.Generator(device="cuda").manual_seed(m)
        w = [torch.randn(128, 768 * 2048, generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.02) for _ in range(3)]
        x = torch.randn(m, 2048, generator=g, device="cuda")
        logits = torch.randn(m, 128, generator=g, device="cuda")
        check_bits(lib, Call(lib, fw, shape_of(fw), w, x, logits, None))


def test_tensors_that_the_binding_refuses(lib):
    fw = F("refuse", W.DT_BF16, 2, 64, 32, 2, 4, 71, 0.05)
    w, shape = weights(fw), shape_of(fw)
    xh, lh, bh = W.ffn_inputs(fw)
    good = Call(lib, fw, shape, w, to_dev(xh), to_dev(lh), to_dev(bh))
    good()
    for change in (dict(x=good.x.cpu()), dict(x=good.x.t()), dict(x=good.x.half()), dict(x=good.x[:1]),
                   dict(ids=good.ids.long()), dict(ids=good.ids[:1]), dict(gates=good.gates[:3]),
                   dict(out=good.out[:100]), dict(logits=good.logits[:1]), dict(bias=good.bias[:3])):
        call = Call(lib, fw, shape, w, good.x, good.logits, good.bias)
        for name, t in change.items():
            setattr(call, name, t)
        with pytest.raises(ValueError):
            call()
    for change in (dict(w=[w[0][:3], w[1], w[2]]), dict(w=[w[0], w[1], w[2][:3]]), dict(scratch=good.scratch[:256])):
        call = Call(lib, fw, shape, w, good.x, good.logits, good.bias)
        for name, t in change.items():
            setattr(call, name, t)
        with pytest.raises(B.EidmError) as e:
            call()
        assert e.value.code == B.E_SIZE
    torch.cuda.synchronize()
