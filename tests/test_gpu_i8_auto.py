"""The route that AUTO takes for 8-bit products and FFNs whose rows of weights
are short: a load of a row by itself takes a whole wavefront's however short."""
import pytest

import i8_cases as I
from expert_id_matmul_amd import binding as B
from test_gpu_ffn_i8 import Ffn
from test_gpu_i8 import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k,top_k,experts,route", [
    (64, 3400, 64, 8, 256, B.GROUPED), (64, 3400, 65, 8, 256, B.GROUPED), (16, 2048, 64, 8, 256, B.GROUPED),
    (32, 1000, 255, 8, 64, B.GROUPED), (1, 2048, 64, 8, 256, B.DIRECT), (8, 1000, 101, 4, 64, B.DIRECT),
    (16, 1000, 1001, 4, 64, B.DIRECT)])
def test_products_of_short_rows(lib, m, n, k, top_k, experts, route):
    c = Call(lib, m, n, k, top_k, experts, False, "mixed")
    assert c(B.AUTO) == route
    I.same(c.result(B.AUTO), c.want())


@pytest.mark.parametrize("m,hidden,inter,top_k,experts,route", [
    (64, 64, 700, 8, 64, B.GROUPED), (64, 1024, 64, 8, 128, B.GROUPED), (2, 64, 700, 8, 64, B.DIRECT),
    (16, 1024, 512, 4, 32, B.DIRECT)])
def test_ffns_of_short_rows(lib, m, hidden, inter, top_k, experts, route):
    c = Ffn(lib, m, hidden, inter, top_k, experts, True, True)
    assert c(B.AUTO) == route
    c.check(c.result(B.AUTO), I.ffn(c.d, top_k, True))
