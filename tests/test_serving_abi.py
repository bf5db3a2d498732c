"""eidm_moe_ffn_decode and eidm_lora_linear on the CPU: sizes and refusals,
all before any launch (no test here touches a GPU)."""
import ctypes

import pytest

from expert_id_matmul_amd import binding as B

FAKE = 0x7F0000000000  # never dereferenced: every call below is refused first


def test_struct_and_constants_match_the_header():
    assert ctypes.sizeof(B.LoraShape) == 56
    text = open(B.__file__.replace("expert_id_matmul_amd/binding.py", "include/eidm.h")).read()
    assert f"#define EIDM_DECODE_MAX_TOKENS {B.DECODE_MAX_TOKENS}\n" in text
    assert f"#define EIDM_LORA_MAX_RANK {B.LORA_MAX_RANK}\n" in text
    assert f"#define EIDM_NO_ADAPTER {hex(B.NO_ADAPTER)}u\n" in text


def ffn(**kw):
    s = B.make_ffn_shape(B.BF16, 4, 64, 32, 2, 8)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_decode_scratch_grows_with_the_rows(lib):
    small, big = lib.moe_ffn_decode_scratch_bytes(ffn(m=1)), lib.moe_ffn_decode_scratch_bytes(ffn(m=64))
    assert 0 < small < big
    assert small >= 2 * 32 * 4 and big >= 64 * 2 * 32 * 4


DECODE = dict(w_gate=FAKE, w_up=FAKE, gu=8 * 64 * 32 * 2, w_down=FAKE, dn=8 * 64 * 32 * 2, x=FAKE, logits=FAKE,
              bias=FAKE, renorm=1, ids=FAKE, gates=FAKE, out=FAKE, scratch=FAKE, sbytes=1 << 20, stream=0)


def decode(lib, shape, **kw):
    a = dict(DECODE, **kw)
    rc = lib.lib.eidm_moe_ffn_decode(ctypes.addressof(shape) if shape is not None else None, *a.values())
    assert lib.last_error()
    d = lib.last_dispatch() if rc == 0 else None
    return rc, d


@pytest.mark.parametrize("field,value,code", [
    ("struct_size", 40, B.E_INVALID), ("m", 0, B.E_INVALID), ("hidden", 0, B.E_INVALID), ("inter", 0, B.E_INVALID),
    ("top_k", 0, B.E_INVALID), ("n_experts", 0, B.E_INVALID), ("weight_dtype", 3, B.E_INVALID),
    ("m", 65, B.E_UNSUPPORTED), ("n_experts", 2049, B.E_UNSUPPORTED), ("top_k", 9, B.E_INVALID),
    ("gate_up_stride_bytes", 4097, B.E_ALIGN), ("down_stride_bytes", 4097, B.E_ALIGN),
    ("gate_up_stride_bytes", 2048, B.E_INVALID), ("down_stride_bytes", 2048, B.E_INVALID)])
def test_decode_refuses_bad_shapes(lib, field, value, code):
    s = ffn(**{field: value})
    assert decode(lib, s)[0] == code
    assert lib.lib.eidm_moe_ffn_decode_scratch_bytes(ctypes.byref(s)) == 0
    with pytest.raises(B.EidmError):
        lib.moe_ffn_decode_scratch_bytes(s)


def test_decode_refuses_more_slots_than_its_limit(lib):
    assert decode(lib, ffn(n_experts=64, top_k=17), gu=1 << 30, dn=1 << 30)[0] == B.E_UNSUPPORTED


@pytest.mark.parametrize("hidden,inter,code", [(32768, 8, 0), (8, 32768, 0), (32769, 8, B.E_UNSUPPORTED),
                                               (8, 32769, B.E_UNSUPPORTED)])
def test_decode_limits_the_length_of_a_row(lib, hidden, inter, code):
    s = B.make_ffn_shape(B.BF16, 3, hidden, inter, 2, 4)
    if code:
        assert decode(lib, s, gu=1 << 40, dn=1 << 40)[0] == code
    assert (lib.lib.eidm_moe_ffn_decode_scratch_bytes(ctypes.byref(s)) == 0) == (code != 0)


@pytest.mark.parametrize("arg", ["w_gate", "w_up", "w_down", "x", "logits", "ids", "gates", "out", "scratch"])
def test_decode_refuses_null_buffers(lib, arg):
    assert decode(lib, ffn(), **{arg: None})[0] == B.E_INVALID


def test_decode_refuses_a_null_shape(lib):
    assert decode(lib, None)[0] == B.E_INVALID


@pytest.mark.parametrize("arg,value,code", [
    ("gu", DECODE["gu"] - 1, B.E_SIZE), ("dn", DECODE["dn"] - 1, B.E_SIZE), ("sbytes", 255, B.E_SIZE),
    ("scratch", FAKE + 128, B.E_ALIGN), ("w_gate", FAKE + 1, B.E_ALIGN), ("w_up", FAKE + 1, B.E_ALIGN),
    ("w_down", FAKE + 1, B.E_ALIGN), ("x", FAKE + 2, B.E_ALIGN), ("logits", FAKE + 1, B.E_ALIGN),
    ("bias", FAKE + 2, B.E_ALIGN), ("ids", FAKE + 2, B.E_ALIGN), ("gates", FAKE + 2, B.E_ALIGN),
    ("out", FAKE + 2, B.E_ALIGN)])
def test_decode_refuses_short_and_misaligned_buffers(lib, arg, value, code):
    assert decode(lib, ffn(), **{arg: value})[0] == code


def lora(**kw):
    s = B.make_lora_shape(B.BF16, B.BF16, 6, 48, 64, 4, 8)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


LORA = dict(w=FAKE, wbytes=48 * 64 * 2, base=None, a=FAKE, abytes=4 * 8 * 64 * 2, b=FAKE, bbytes=4 * 8 * 48 * 2,
            ranks=FAKE, scales=FAKE, x=FAKE, ids=FAKE, out=FAKE, scratch=FAKE, sbytes=1 << 24, stream=0)


def linear(lib, shape, **kw):
    a = dict(LORA, **kw)
    rc = lib.lib.eidm_lora_linear(ctypes.addressof(shape) if shape is not None else None, *a.values())
    assert lib.last_error()
    return rc


@pytest.mark.parametrize("field,value,code", [
    ("struct_size", 48, B.E_INVALID), ("m", 0, B.E_INVALID), ("n", 0, B.E_INVALID), ("k", 0, B.E_INVALID),
    ("n_adapters", 0, B.E_INVALID), ("max_rank", 0, B.E_INVALID), ("weight_dtype", 3, B.E_INVALID),
    ("adapter_dtype", 9, B.E_INVALID), ("arith", 2, B.E_INVALID), ("max_rank", 257, B.E_INVALID),
    ("n_adapters", 2049, B.E_UNSUPPORTED), ("m", 2 ** 31, B.E_UNSUPPORTED),
    ("a_stride_bytes", 1025, B.E_ALIGN), ("b_stride_bytes", 769, B.E_ALIGN),
    ("a_stride_bytes", 1022, B.E_INVALID), ("b_stride_bytes", 766, B.E_INVALID),
    ("a_stride_bytes", 2 ** 63, B.E_INVALID)])
def test_lora_refuses_bad_shapes(lib, field, value, code):
    s = lora(**{field: value})
    assert linear(lib, s) == code
    assert lib.lib.eidm_lora_linear_scratch_bytes(ctypes.byref(s)) == 0
    with pytest.raises(B.EidmError):
        lib.lora_linear_scratch_bytes(s)


def test_lora_refuses_ranks_above_its_limit(lib):
    s = B.make_lora_shape(B.BF16, B.BF16, 6, 48, 64, 4, 257)
    assert linear(lib, s, abytes=1 << 30, bbytes=1 << 30) == B.E_UNSUPPORTED


def test_lora_refuses_a_grid_beyond_a_launch(lib):
    s = B.make_lora_shape(B.BF16, B.BF16, 1 << 26, 1 << 18, 8, 4, 8)
    assert linear(lib, s, abytes=1 << 40, bbytes=1 << 40, wbytes=1 << 40) == B.E_UNSUPPORTED


def test_lora_reads_no_weight_dtype_beside_a_base(lib):
    s = lora(weight_dtype=77, arith=5)
    assert linear(lib, s, w=None, base=FAKE, sbytes=255) == B.E_SIZE  # past the shape's checks


def test_lora_takes_weights_or_base_and_not_both(lib):
    assert linear(lib, lora(), base=FAKE) == B.E_INVALID
    assert linear(lib, lora(), w=None) == B.E_INVALID


@pytest.mark.parametrize("arg", ["a", "b", "x", "ids", "out", "scratch"])
def test_lora_refuses_null_buffers(lib, arg):
    assert linear(lib, lora(), **{arg: None}) == B.E_INVALID


def test_lora_refuses_a_null_shape(lib):
    assert linear(lib, None) == B.E_INVALID


@pytest.mark.parametrize("arg,value,code", [
    ("wbytes", LORA["wbytes"] - 1, B.E_SIZE), ("abytes", LORA["abytes"] - 1, B.E_SIZE),
    ("bbytes", LORA["bbytes"] - 1, B.E_SIZE), ("sbytes", 255, B.E_SIZE), ("scratch", FAKE + 64, B.E_ALIGN),
    ("w", FAKE + 1, B.E_ALIGN), ("a", FAKE + 1, B.E_ALIGN), ("b", FAKE + 1, B.E_ALIGN), ("x", FAKE + 2, B.E_ALIGN),
    ("ranks", FAKE + 2, B.E_ALIGN), ("scales", FAKE + 1, B.E_ALIGN), ("ids", FAKE + 2, B.E_ALIGN),
    ("out", FAKE + 2, B.E_ALIGN)])
def test_lora_refuses_short_and_misaligned_buffers(lib, arg, value, code):
    assert linear(lib, lora(), **{arg: value}) == code


def test_lora_refuses_a_misaligned_base(lib):
    assert linear(lib, lora(), w=None, base=FAKE + 2) == B.E_ALIGN


def test_lora_split16_keeps_that_arithmetics_conditions(lib):
    s = B.make_lora_shape(B.BF16, B.BF16, 6, 48, 60, 4, 8, arith=B.ARITH_SPLIT16)  # k not a multiple of 8
    assert linear(lib, s) == B.E_UNSUPPORTED
    s = B.make_lora_shape(B.F32, B.BF16, 6, 48, 64, 4, 8, arith=B.ARITH_SPLIT16)
    assert linear(lib, s) == B.E_UNSUPPORTED
    s = lora(arith=B.ARITH_SPLIT16)
    assert linear(lib, s, x=FAKE + 4) == B.E_ALIGN
    assert linear(lib, s, w=FAKE + 8) == B.E_ALIGN


# HIP takes fewer than 2^32 threads a launch: 2^24 blocks of 256
@pytest.mark.parametrize("m,n,k,adapters,max_rank,code", [
    (1 << 25, 64, 64, 4, 256, B.E_UNSUPPORTED),          # the shrink's blocks: 32 ranks each
    ((1 << 25) - 16 * 6, 64, 64, 4, 256, 0),
    (1, 8188 * 256 + 1, 16385, 2048, 1, B.E_UNSUPPORTED),  # the expand's: 256 columns each, many adapters
    (1, 8188 * 256, 16385, 2048, 1, 0),
    (1, 1 << 29, 8, 2, 4, B.E_UNSUPPORTED),              # the projection of one row
    (1, (1 << 29) - 16, 8, 2, 4, 0)])
def test_lora_grids_stay_below_a_launchs_threads(lib, m, n, k, adapters, max_rank, code):
    s = B.make_lora_shape(B.BF16, B.BF16, m, n, k, adapters, max_rank)
    assert linear(lib, s, abytes=1 << 50, bbytes=1 << 50, wbytes=1 << 50, sbytes=0) == (code or B.E_SIZE)
    assert (lib.lib.eidm_lora_linear_scratch_bytes(ctypes.byref(s)) == 0) == (code != 0)


def test_lora_one_row_on_a_base_has_no_projection_to_refuse(lib):
    s = B.make_lora_shape(B.BF16, B.BF16, 1, 1 << 29, 8, 2, 4)
    assert linear(lib, s, w=None, base=FAKE, abytes=1 << 50, bbytes=1 << 50, sbytes=0) == B.E_SIZE
