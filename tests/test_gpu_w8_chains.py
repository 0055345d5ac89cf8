"""Products in a row without a pause, where what one leaves behind could meet the next."""
import threading

import pytest
import torch

import fractional_bit_weight_b200 as lq
import w8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def operands(batch, K, N, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = [torch.zeros(r, lq.i8_row_bytes(K), dtype=torch.int8, device=DEV) for r in (batch, N)]
    for t in q:
        t[:, :K] = torch.randint(-127, 128, (t.shape[0], K), generator=g, device=DEV).to(torch.int8)
    s = [torch.rand(r, generator=g, device=DEV) * 0.02 + 1e-3 for r in (batch, N)]
    return q[0], s[0], q[1], s[1]


ROUTES = [lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR, lq.I8_ROUTE_SPLIT]


@pytest.mark.parametrize("other", ROUTES)
@pytest.mark.parametrize("batch,K,N", [(40, 256, 1000), (300, 1000, 4104), (513, 4096, 2050)])
def test_pairs_leave_nothing_behind(batch, K, N, other):
    """The odd CTA of a pair waits for the even one's last commits. What follows on its SM has live
    barriers at the same places: a late arrival there would let a stage through too early."""
    ws = lq.new_i8_workspace()
    first, second = operands(batch, K, N, 1), operands(batch + 9, K + 128, N, 2)
    want = [lq.gemm_i8(*first, K=K, dtype=BF16, workspace=ws, route=lq.I8_ROUTE_PAIR),
            lq.gemm_i8(*second, K=K + 128, workspace=ws, route=other)]
    for got, ops, k in zip(want, (first, second), (K, K + 128)):
        ref.within(got, *ref.product(*ops, k, None))
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for _ in range(6):
            got.append(lq.gemm_i8(*first, K=K, dtype=BF16, workspace=ws, route=lq.I8_ROUTE_PAIR))
            got.append(lq.gemm_i8(*second, K=K + 128, workspace=ws, route=other))
        for i, y in enumerate(got):
            assert torch.equal(y, want[i % 2])
    assert lq.device_status(ws) == (lq.LQ_OK, 0)


def test_clusters_on_two_streams():
    """Small clusters of two and eight CTAs from two streams at once."""
    ws = lq.new_i8_workspace()
    shapes = [(164, 1024, 8), (1025, 256, 24), (40, 256, 1000), (200, 384, 520)]
    routes = [None, None, lq.I8_ROUTE_PAIR, lq.I8_ROUTE_SPLIT]
    ops = [operands(*s, seed=i) for i, s in enumerate(shapes)]
    want = [lq.gemm_i8(*o, K=s[1], workspace=ws, route=r) for o, s, r in zip(ops, shapes, routes)]
    for y, o, s in zip(want, ops, shapes):
        ref.within(y, *ref.product(*o, s[1], None))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for _ in range(4):
            for i, (o, s, r) in enumerate(zip(ops, shapes, routes)):
                with torch.cuda.stream(streams[i % 2]):
                    got.append(lq.gemm_i8(*o, K=s[1], workspace=ws, route=r))
        torch.cuda.synchronize()
        for i, y in enumerate(got):
            assert torch.equal(y, want[i % 4])
    assert lq.device_status(ws) == (lq.LQ_OK, 0)


def test_two_host_threads():
    """Calls of different shapes from two threads, each on its own stream."""
    ws = lq.new_i8_workspace()
    shapes = [[(2, 512, 300), (40, 256, 1000), (300, 1000, 4104), (33, 8192, 40)],
              [(130, 128, 64), (16, 1000, 260), (20, 8192, 1024), (513, 256, 1030)]]
    ops = [[operands(*s, seed=10 * t + i) for i, s in enumerate(shapes[t])] for t in range(2)]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(t):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[t] = [lq.gemm_i8(*o, K=s[1], workspace=ws)
                              for o, s in zip(ops[t], shapes[t])]
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # noqa: BLE001 (reported below, in the test's own thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for t in range(2):
        for y, o, s in zip(got[t], ops[t], shapes[t]):
            ref.within(y, *ref.product(*o, s[1], None))
    assert lq.device_status(ws) == (lq.LQ_OK, 0)
