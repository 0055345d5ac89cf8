"""The tile plans of lq_gemm_i8 (host-only query): what fits an SM, and what must not share one."""
import itertools

import pytest

import fractional_bit_weight_b200 as lq
from fractional_bit_weight_b200 import build as lqbuild

SM_SMEM = 228 * 1024        # shared memory of an SM; each resident CTA takes 1 KB more than it asks
CTA_SMEM = 227 * 1024       # the most one CTA can have
BATCHES = (1, 3, 16, 17, 33, 64, 100, 129, 164, 256, 300, 513, 1025, 2049, 4096, 70000)
INPUTS = (1, 17, 128, 129, 256, 640, 1024, 2056, 4096, 8192, 14337, 28672, 131071)
ROWS = (1, 8, 24, 129, 257, 441, 1024, 1184, 4104, 8192, 28672)
TILE_ROUTES = (None, lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR, lq.I8_ROUTE_SPLIT)


@pytest.fixture(scope="module", autouse=True)
def built():
    lqbuild.build()


def sweep(routes):
    for batch, K, N, route in itertools.product(BATCHES, INPUTS, ROWS, routes):
        yield (batch, K, N, route), lq.gemm_i8_plan(batch, K, N, route)


def test_clusters_have_their_sms_to_themselves():
    """A CTA of a cluster holds tensor memory while it waits for its peers to get theirs: two such
    CTAs on one SM could wait for each other's clusters."""
    seen = set()
    for shape, p in sweep(TILE_ROUTES):
        assert p["smem"] <= CTA_SMEM, (shape, p)
        if p["cluster"] > 1:
            seen.add((p["route"], p["cluster"]))
            assert 2 * (p["smem"] + 1024) > SM_SMEM, (shape, p)
    assert seen == {(lq.I8_ROUTE_PAIR, 2), (lq.I8_ROUTE_SPLIT, 2), (lq.I8_ROUTE_SPLIT, 4),
                    (lq.I8_ROUTE_SPLIT, 8)}


@pytest.mark.parametrize("batch,K,N,cluster", [(164, 1024, 8, 8), (1025, 256, 24, 2)])
def test_small_clusters_of_the_own_choice(batch, K, N, cluster):
    """Layers whose clusters need little shared memory for their operands."""
    p = lq.gemm_i8_plan(batch, K, N)
    assert lq.gemm_i8_route(batch, K, N) == p["route"] == lq.I8_ROUTE_SPLIT
    assert p["cluster"] == cluster and 2 * (p["smem"] + 1024) > SM_SMEM


def test_tiles_cover_the_call():
    for (batch, K, N, route), p in sweep(TILE_ROUTES):
        if route is not None:
            assert p["route"] == route
        ctas = 2 if p["route"] == lq.I8_ROUTE_PAIR else 1
        assert 8 <= p["rows"] <= 128 and p["rows"] % 8 == 0
        assert 16 <= p["tokens"] <= 256 and p["tokens"] % (16 * ctas) == 0
        assert p["tiles"] == -(-N // (p["rows"] * ctas)) * -(-batch // p["tokens"])
        assert p["stages"] >= 4 and p["chunks"] >= 1


def test_plan_refusals():
    for bad in ((0, 64, 64, None), (1, 0, 64, None), (1, 64, 0, None), (1, 131072, 64, None),
                (1, 64, 64, lq.I8_ROUTE_GEMV), (1, 64, 64, 4), (1, 64, 64, -2)):
        with pytest.raises(lq.LQError):
            lq.gemm_i8_plan(*bad)
    assert lq.lib().lq_gemm_i8_plan(1, 64, 64, -1, None) == lq.LQ_EINVAL


def test_second_wave_of_the_gemv():
    """Long rows leave the GEMV where its CTAs of 16 rows are more than 8 on each of the 148 SMs."""
    edge = 16 * 8 * 148
    for batch in (1, 4, 8):
        for K in (8192, 10240, 28672):
            assert lq.gemm_i8_route(batch, K, edge) == lq.I8_ROUTE_GEMV
            assert lq.gemm_i8_route(batch, K, edge + 1) != lq.I8_ROUTE_GEMV
        assert lq.gemm_i8_route(batch, 4096, 2 * edge) == lq.I8_ROUTE_GEMV
