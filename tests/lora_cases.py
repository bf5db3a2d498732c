"""Seeded adapter problems for the lora_linear tests, their evaluation in the
documented order on the CPU, and a per-element error bound."""
from __future__ import annotations

import ctypes
import os
import subprocess
from dataclasses import dataclass

import numpy as np
import torch

from expert_id_matmul_amd import workloads as W
from helpers import canonical_matmul_id, host_threads

HERE = os.path.dirname(os.path.abspath(__file__))
NO_ADAPTER = 0xFFFFFFFF
TORCH = {W.DT_F32: torch.float32, W.DT_F16: torch.float16, W.DT_BF16: torch.bfloat16}
U = 2.0 ** -24  # f32 rounding: half a step, relative


@dataclass(frozen=True)
class Lora:
    """runs: the rows are that many runs of consecutive rows with one adapter
    each, 0: an adapter per row.  pad: scalars between adapters of A and of B."""

    name: str
    w_dtype: int
    a_dtype: int
    m: int
    n: int
    k: int
    n_adapters: int
    max_rank: int
    runs: int = 0
    ranks: bool = True
    scales: bool = True
    given: bool = False
    pad: int = 0
    arith: int = 0
    none: float = 0.2
    seed: int = 1

    @property
    def a_stride(self) -> int:
        return (self.max_rank * self.k + self.pad) * W.DTYPE_SIZE[self.a_dtype]

    @property
    def b_stride(self) -> int:
        return (self.n * self.max_rank + self.pad) * W.DTYPE_SIZE[self.a_dtype]

    def workload(self, n: int, k: int, experts: int, dtype: int, stride: int) -> W.Workload:
        """One row-selected product of this problem as a matmul_id workload."""
        return W.Workload(self.name, dtype, self.m, n, k, 1, experts, stride, W.LAYOUT_SHARED, W.IDS_DISTINCT,
                          self.seed, 1.0, "random", "uniform")


def _bytes(t: torch.Tensor) -> np.ndarray:
    return t.contiguous().view(torch.uint8).numpy().reshape(-1).copy()


def _stack(t: torch.Tensor, pad: int) -> np.ndarray:
    """[adapters, ...] as bytes with `pad` scalars (NaN) after each adapter."""
    flat = t.reshape(t.shape[0], -1)
    if pad:
        flat = torch.cat([flat, torch.full((t.shape[0], pad), float("nan"), dtype=t.dtype)], 1)
    return _bytes(flat)


def inputs(p: Lora) -> dict:
    g = torch.Generator().manual_seed(p.seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    d = {"x": rnd(p.m, p.k).numpy(),
         "w": None if p.given else _bytes((rnd(p.n, p.k) * p.k ** -0.5).to(TORCH[p.w_dtype])),
         "base": rnd(p.m, p.n).numpy() if p.given else None}
    a = (rnd(p.n_adapters, p.max_rank, p.k) * p.k ** -0.5).to(TORCH[p.a_dtype])
    b = (rnd(p.n_adapters, p.n, p.max_rank) * p.max_rank ** -0.5).to(TORCH[p.a_dtype])
    d["a"], d["b"], d["b32"] = _stack(a, p.pad), _stack(b, p.pad), b.float().numpy()
    d["ranks"] = d["scales"] = None
    if p.ranks:  # 0 .. max_rank, with values above max_rank, which count as max_rank
        r = torch.randint(0, p.max_rank + 1, (p.n_adapters,), generator=g)
        r[torch.rand(p.n_adapters, generator=g) < 0.2] = 1 << 20
        d["ranks"] = r.numpy().astype(np.uint32)
    if p.scales:
        d["scales"] = rnd(p.n_adapters).numpy()
    per = p.runs or p.m
    ids = torch.randint(0, p.n_adapters, (per,), generator=g)
    ids[torch.rand(per, generator=g) < p.none] = NO_ADAPTER
    if p.runs:
        cuts = torch.randint(0, p.m + 1, (per - 1,), generator=g).sort().values
        ids = ids[torch.searchsorted(cuts, torch.arange(p.m), right=True)]
    d["ids"] = ids.numpy().astype(np.uint32)
    return d


_lib = None


def _expand_lib():
    global _lib
    if _lib is None:
        src, so = os.path.join(HERE, "canonical_lora.c"), os.path.join(HERE, "_canonical_lora.so")
        if not os.path.exists(so) or os.path.getmtime(so) < os.path.getmtime(src):
            subprocess.run(["gcc", "-O2", "-std=c11", "-fPIC", "-shared", "-ffp-contract=off", "-fno-fast-math", src,
                            "-o", so + ".tmp", "-lm"], check=True)
            os.replace(so + ".tmp", so)
        _lib = ctypes.CDLL(so)
        P, u32 = ctypes.c_void_p, ctypes.c_uint32
        _lib.canonical_lora_expand.argtypes = [u32, u32, u32, u32, u32, P, P, P, P, P, P, P]
    return _lib


def base_bits(p: Lora, d: dict) -> np.ndarray:
    """The shared projection in the documented f32 order, or the given rows."""
    if p.given:
        return d["base"]
    wl = p.workload(p.n, p.k, 1, p.w_dtype, p.n * p.k * W.DTYPE_SIZE[p.w_dtype])
    return canonical_matmul_id(wl, d["w"], d["x"], np.zeros((p.m, 1), np.uint32), threads=host_threads())


def documented(p: Lora, d: dict, base: np.ndarray) -> np.ndarray:
    """out f32 [m, n] in the documented order, from the base rows' bits."""
    wl = p.workload(p.max_rank, p.k, p.n_adapters, p.a_dtype, p.a_stride)
    v = canonical_matmul_id(wl, d["a"], d["x"], d["ids"].reshape(-1, 1), threads=host_threads())
    base = np.ascontiguousarray(base, np.float32)
    out = np.empty((p.m, p.n), np.float32)
    ptr = lambda z: None if z is None else np.ascontiguousarray(z).ctypes.data_as(ctypes.c_void_p)
    b32 = np.ascontiguousarray(d["b32"])
    _expand_lib().canonical_lora_expand(p.m, p.n, p.n_adapters, p.max_rank, p.max_rank, ptr(base), ptr(b32),
                                        ptr(d["ranks"]), ptr(d["scales"]), ptr(v), ptr(d["ids"]), ptr(out))
    return out


def widened(raw: np.ndarray, dtype: int) -> np.ndarray:
    return torch.from_numpy(raw.copy()).view(TORCH[dtype]).double().numpy()


def bound(p: Lora, d: dict) -> np.ndarray:
    """Per element, the most that f32 rounding allows between out and its
    64-bit value: a k-term product in 16 slices of k/16 fused steps and a
    4-level tree is off by at most (k/16 + 4) U sum |w x| to first order (1%
    is added for the rest), u by rank steps on top of v's error, and and
    the scale-and-add rounds once."""
    k, r = p.k, p.max_rank
    ck = (k + 127) // 128 * 8 + 4
    x = np.abs(d["x"].astype(np.float64))
    e = np.zeros((p.m, p.n))
    mag = np.abs(d["base"].astype(np.float64)) if p.given else None
    if not p.given:
        mag = x @ np.abs(widened(d["w"], p.w_dtype).reshape(p.n, k)).T
        e = ck * U * mag
    a = widened(d["a"], p.a_dtype).reshape(p.n_adapters, -1)[:, : r * k].reshape(p.n_adapters, r, k)
    for i in np.unique(d["ids"]):
        if i >= p.n_adapters:
            continue
        t = np.nonzero(d["ids"] == i)[0]
        live = r if d["ranks"] is None else min(int(d["ranks"][i]), r)
        s = 1.0 if d["scales"] is None else abs(float(d["scales"][i]))
        um = (x[t] @ np.abs(a[i, :live]).T) @ np.abs(d["b32"][i, :, :live].astype(np.float64)).T
        e[t] += s * um * (ck + live + 1) * U
        mag[t] += s * um
    return 1.01 * (e + U * mag) + 1e-37
