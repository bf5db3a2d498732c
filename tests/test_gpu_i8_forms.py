"""Each form of the 8-bit tiles (launch_i8_tiles: the tile by the rows of an
expert and by what fills the device) bit for bit against the definition, with
several steps of k of which the last is partial, more than eight row tiles of
one expert where the rule's average allows it, rows whose ids name no expert,
and the form that ran told by the launch receipt."""
import numpy as np
import pytest
import torch

import i8_cases as I
from expert_id_matmul_amd import binding as B
from helpers import ids_to_dev, to_dev
from test_gpu_ffn_i8 import Ffn
from test_gpu_i8 import Call

pytestmark = pytest.mark.gpu

WHOLE, ODD = 272, 259  # k: rows of whole 16 bytes go straight into LDS, others through registers

# rows x columns of a tile: threads of a block, steps of k that the LDS holds
FORMS = {(32, 64): (256, 3), (32, 128): (256, 2), (64, 128): (256, 2), (128, 128): (512, 2), (256, 256): (512, 2)}


def launched(lib, kernel):
    d = lib.last_dispatch()
    (at,) = [i for i, name in enumerate(d.kernels()) if name == kernel]
    return d.launches[at].block, d.launches[at].lds_bytes


def form(tile, k, experts):
    """Block and LDS bytes; experts None: one weight without ids."""
    threads, stages = FORMS[tile]
    ids = 0 if experts is None else (experts + 2) * 8
    return threads, (stages if k % 16 == 0 else 2) * sum(tile) * 128 + ids


# tile, experts, m, top_k, n, rows of expert 0 of m * top_k (the others take the rest in turn)
BY_IDS = {
    "32x64": ((32, 64), 5, 300, 2, 200, 0.6),
    "32x128": ((32, 128), 16, 100, 3, 2050, 0.1),
    "64x128": ((64, 128), 8, 160, 2, 4100, 0.2),
    "128x128": ((128, 128), 4, 610, 2, 2900, 0.9),
    "256x256": ((256, 256), 2, 1210, 2, 6700, 0.96),
    # weights of 64 MB and more: an expert's past the caches where one tile alone reads them
    "32x128 past the caches": ((32, 128), 128, 400, 4, 2050, 0.03),
    "64x128 past the caches": ((64, 128), 64, 900, 2, 4100, 0.06),
}


@pytest.mark.parametrize("k", [WHOLE, ODD], ids=["straight", "registers"])
@pytest.mark.parametrize("slotted", [False, True], ids=["shared", "slotted"])
@pytest.mark.parametrize("name", BY_IDS)
def test_tiles_by_ids(lib, name, k, slotted):
    tile, experts, m, top_k, n, share = BY_IDS[name]
    c = Call(lib, m, n, k, top_k, experts, slotted, "mixed")
    g = np.random.default_rng(m + k)
    flat = 1 + g.integers(0, experts - 1, m * top_k)
    flat[g.random(m * top_k) < share] = 0
    flat[[3, 17, m * top_k - 1]] = experts, 0xFFFFFFFF, experts  # no expert's
    c.ids[:] = flat.reshape(m, top_k)
    c.dids = ids_to_dev(c.ids)
    assert ("past" in name) == (experts * n * k >= 64_000_000)
    got = c.result(B.GROUPED)
    assert launched(lib, "i8_tiles") == form(tile, k, experts)
    I.same(got, c.want(), name)


ONE = {
    "32x64": ((32, 64), 100, 1000),
    "32x128": ((32, 128), 20, 33000),
    "64x128": ((64, 128), 48, 33000),
    "128x128": ((128, 128), 1300, 3000),
    "256x256": ((256, 256), 4000, 4200),
}


@pytest.mark.parametrize("k", [WHOLE, ODD], ids=["straight", "registers"])
@pytest.mark.parametrize("name", ONE)
def test_tiles_of_one_weight(lib, name, k):
    tile, m, n = ONE[name]
    c = Call(lib, m, n, k, 1, 1, False, "mixed", dense=True)
    got = c.result(B.GROUPED)
    assert launched(lib, "i8_tiles") == form(tile, k, None)
    I.same(got, c.want(), name)


# tile, experts, m, top_k, inter, what expert 0's logits have more
GATE_UP = {
    "32x64": ((32, 64), 5, 300, 2, 90, 2.0),
    "32x128": ((32, 128), 16, 100, 3, 1030, 0.5),
    "64x128": ((64, 128), 8, 160, 2, 2060, 0.5),
    "128x128": ((128, 128), 4, 610, 2, 1450, 4.0),
    "256x256": ((256, 256), 2, 2450, 1, 3400, 4.0),
    "32x128 past the caches": ((32, 128), 128, 400, 4, 1030, 0.5),
    "64x128 past the caches": ((64, 128), 64, 900, 2, 2060, 1.0),
}


@pytest.mark.parametrize("hidden", [WHOLE, ODD], ids=["straight", "registers"])
@pytest.mark.parametrize("name", GATE_UP)
def test_gate_and_up_tiles(lib, name, hidden):
    tile, experts, m, top_k, inter, more = GATE_UP[name]
    c = Ffn(lib, m, hidden, inter, top_k, experts, False, True)
    c.d["logits"][:, 0] += np.float32(more)
    c.logits = to_dev(c.d["logits"])
    assert ("past" in name) == (experts * 2 * inter * hidden >= 64_000_000)
    got = c.result(B.GROUPED)
    assert launched(lib, "i8_gate_up_tiles") == form(tile, hidden, experts)
    c.check(got, I.ffn(c.d, top_k, True))


def test_rows_off_16_bytes_go_through_registers(lib):
    """Whole rows from an address or at a distance that is no multiple of 16: LDS holds two steps, not three."""
    for pad, shift in ((0, 0), (16, 0), (8, 0), (0, 4)):
        c = Call(lib, 60, 90, 256, 2, 3, False, "mixed", pad=pad, shift=shift)
        got = c.result(B.GROUPED)
        steps = 3 if pad % 16 == 0 and shift % 16 == 0 else 2
        assert launched(lib, "i8_tiles") == (256, steps * 96 * 128 + 5 * 8)
        I.same(got, c.want())
