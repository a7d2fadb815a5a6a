"""CPU-only: the plan queries of the 8-bit product and of the orthogonalisation, and that plans.py has a
shape for every plan there is."""
import math
import random

import pytest

import dense_fp32_matrix_08_gb300 as sg
from plans import ORTHOGONALIZATIONS, PRODUCTS

SMS = 152


def product_key(M, N, K, ta, tb, ar, bc):
    p = sg.f8_gemm_plan(M, N, K, transa=ta, transb=tb, a_rows=ar, b_cols=bc, num_sms=SMS)
    return (int(p["exchanged"]), p["tile_cols"], p["split"])


def storage(key, shape):
    """How P and Q of a product are stored, and whether Q has a scale for each column."""
    *_, ta, tb, ar, bc = shape
    return key, ta, tb, (ar if key[0] else bc) == 1


def orthogonalize_key(batch, m, n):
    p = sg.ns_orthogonalize_plan(batch, m, n, SMS)
    return p["tile_cols"], "".join("-" if s == 1 else "a" if w == 0 else "r"
                                   for s, w in zip(p["split"], p["whole"]))


def test_shapes_have_their_plans():
    for key, shapes in PRODUCTS.items():
        for shape in shapes:
            assert product_key(*shape) == key, shape
    for key, (batch, m, n) in ORTHOGONALIZATIONS.items():
        assert orthogonalize_key(batch, m, n) == key and orthogonalize_key(batch, n, m) == key


def log_uniform(rng, high):
    return int(math.exp(rng.uniform(0, math.log(high))))


def test_no_plan_of_the_product_is_missing():
    have = {storage(k, s) for k, shapes in PRODUCTS.items() for s in shapes}
    rng = random.Random(1)
    for _ in range(60000):
        shape = (log_uniform(rng, 6000), log_uniform(rng, 8000), log_uniform(rng, 8192),
                 rng.randrange(2), rng.randrange(2), rng.choice((1, 128)), rng.choice((1, 128)))
        key = product_key(*shape)
        assert storage(key, shape) in have, (key, shape)


def test_no_plan_of_the_orthogonalisation_is_missing():
    rng = random.Random(2)
    for _ in range(20000):
        batch, m, n = rng.choice((1, 1, 2, 3, 5, 8, 17)), log_uniform(rng, 4200), log_uniform(rng, 17000)
        key = orthogonalize_key(batch, m, n)
        assert key in ORTHOGONALIZATIONS, (key, batch, m, n)


@pytest.mark.parametrize("change,code", [
    (dict(transa=2), -1), (dict(transb=-1), -2), (dict(M=0), -3), (dict(N=0), -4), (dict(K=0), -5),
    (dict(a_rows=2), -6), (dict(b_cols=0), -7), (dict(sms=-1), -8)])
def test_product_refusals(change, code):
    args = dict(transa=0, transb=0, M=4, N=4, K=4, a_rows=1, b_cols=128, sms=0)
    assert sg.lib.f8_gemm_plan(*{**args, **change}.values(), None, None, None) == code
    assert sg.lib.f8_gemm_plan(*args.values(), None, None, None) == 0


@pytest.mark.parametrize("change,code", [
    (dict(batch=0), -1), (dict(rows=0), -2), (dict(cols=0), -3), (dict(sms=-1), -4)])
def test_orthogonalize_refusals(change, code):
    args = dict(batch=1, rows=4, cols=4, sms=0)
    assert sg.lib.ns_orthogonalize_plan(*{**args, **change}.values(), None, None, None, None) == code
    assert sg.lib.ns_orthogonalize_plan(*args.values(), None, None, None, None) == 0


def test_parts_of_a_plan_fit():
    """Tiles computed whole are whole rounds of the GPU's blocks, and the parts of the others at most
    one."""
    rng = random.Random(3)
    for _ in range(2000):
        batch, m, n = rng.choice((1, 2, 8)), log_uniform(rng, 4200), log_uniform(rng, 17000)
        p = sg.ns_orthogonalize_plan(batch, m, n, SMS)
        at_once = SMS // 2 if p["tile_cols"] == 256 else SMS
        for tiles, whole, split in zip(p["tiles"], p["whole"], p["split"]):
            assert 0 <= whole <= tiles and 1 <= split <= 16
            assert whole == tiles if split == 1 else (
                whole % at_once == 0 and (tiles - whole) * split <= at_once)
    with pytest.raises(sg.SgemmError):
        sg.f8_gemm_plan(0, 1, 1)
