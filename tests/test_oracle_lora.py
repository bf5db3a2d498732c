"""The adapters' oracle and the CPU evaluation of their documented order,
pinned to a numpy float64 brute force (library decoders)."""
import numpy as np
import pytest

import oracle
from expert_id_matmul_amd import workloads as W
from lora_cases import NO_ADAPTER, Lora, base_bits, bound, documented, inputs, widened

CASES = [Lora("bf16", W.DT_BF16, W.DT_BF16, 7, 19, 37, 4, 5),
         Lora("f16_f32_padded", W.DT_F16, W.DT_F32, 5, 9, 130, 3, 11, pad=3, scales=False),
         Lora("f32_plain", W.DT_F32, W.DT_F16, 6, 33, 16, 2, 1, ranks=False),
         Lora("given_runs", W.DT_F32, W.DT_BF16, 40, 12, 64, 5, 8, runs=6, given=True, none=0.4)]


def _oracle(p, d):
    return oracle.lora_linear(p.w_dtype, p.a_dtype, p.m, p.n, p.k, p.n_adapters, p.max_rank, p.a_stride, p.b_stride,
                              d["w"], d["base"], d["a"], d["b"], d["ranks"], d["scales"], d["x"], d["ids"])


def _brute(p, d):
    r = p.max_rank
    a = widened(d["a"], p.a_dtype).reshape(p.n_adapters, -1)[:, : r * p.k].reshape(p.n_adapters, r, p.k)
    b = widened(d["b"], p.a_dtype).reshape(p.n_adapters, -1)[:, : p.n * r].reshape(p.n_adapters, p.n, r)
    x = d["x"].astype(np.float64)
    y = d["base"].astype(np.float64) if p.given else x @ widened(d["w"], p.w_dtype).reshape(p.n, p.k).T
    for t, i in enumerate(d["ids"]):
        if i == NO_ADAPTER:
            continue
        live = r if d["ranks"] is None else min(int(d["ranks"][i]), r)
        s = 1.0 if d["scales"] is None else float(d["scales"][i])
        y[t] += s * (b[i, :, :live] @ (a[i, :live] @ x[t]))
    return y


@pytest.mark.parametrize("p", CASES, ids=lambda p: p.name)
def test_oracle_equals_the_brute_force(p):
    d = inputs(p)
    np.testing.assert_allclose(_oracle(p, d), _brute(p, d), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("p", CASES, ids=lambda p: p.name)
def test_documented_order_is_within_the_derived_bound(p):
    d = inputs(p)
    err = np.abs(documented(p, d, base_bits(p, d)).astype(np.float64) - _oracle(p, d))
    assert (err <= bound(p, d)).all()


def test_rows_without_an_adapter_and_with_a_bad_id():
    p = CASES[0]
    d = inputs(p)
    d["ids"][:3] = [NO_ADAPTER, p.n_adapters, 2]
    d["ranks"][2] = 0
    y = _oracle(p, d)
    plain = d["x"].astype(np.float64) @ widened(d["w"], p.w_dtype).reshape(p.n, p.k).T
    np.testing.assert_allclose(y[[0, 2]], plain[[0, 2]], rtol=1e-12)
    assert np.isnan(y[1]).all() and np.isfinite(np.delete(y, 1, 0)).all()


def test_oracle_needs_exactly_one_of_weights_and_base():
    p = CASES[0]
    d = inputs(p)
    with pytest.raises(ValueError):
        _oracle(p, dict(d, base=np.zeros((p.m, p.n))))
    with pytest.raises(ValueError):
        _oracle(p, dict(d, w=None))
