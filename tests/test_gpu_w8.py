"""lq_quant_i8 and lq_gemm_i8 against their definitions in 64 bits."""
import ctypes

import pytest
import torch

import fractional_bit_weight_b200 as lq
import w8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def rand(rows, K, dtype, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(rows, K, generator=g, device=DEV)).to(dtype)


def signs(K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(0, 2, (K,), generator=g, device=DEV).to(torch.int8) * 2 - 1


def check_exact(x, q, scale, values):
    """Without T every code and scale is the definition's."""
    K = x.shape[1]
    want, ws = ref.codes(x.double())
    assert torch.equal(q[:, :K].double(), want)
    assert not q[:, K:].any()
    a = x.float().abs().amax(1)
    bad = ~torch.isfinite(x.float()).all(1)
    # the fp32 quotient, through fp64 (whose 53 bits make the second rounding harmless): torch
    # divides an fp32 tensor by a number as a product with its reciprocal
    s32 = torch.where(bad, torch.full_like(a, float("nan")), (a.double() / 127).float())
    assert torch.equal(torch.isnan(scale), bad)
    assert torch.equal(scale[~bad], s32[~bad])
    v = (want.float() * s32[:, None]).to(x.dtype)
    assert torch.equal(values[~bad], v[~bad]) and torch.isnan(values[bad]).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (2, 16), (5, 100), (4, 256), (1, 264),
                                    (300, 264), (301, 1001), (2, 4097), (3, 8192), (700, 520),
                                    (1, 16384), (2, 28672), (1, 32776), (2, 65536), (1, 65535)])
def test_quant_exact(rows, K, dtype):
    x = rand(rows, K, dtype, rows * 7 + K)
    x[0, K // 2] = 0.0
    q, scale, values = lq.quant_i8(x, values=True)
    assert q.shape == (rows, lq.i8_row_bytes(K)) and values.dtype == dtype
    check_exact(x, q, scale, values)
    q2, scale2 = lq.quant_i8(x)
    assert torch.equal(q, q2) and torch.equal(scale, scale2)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("K", [512, 509])
def test_quant_ties(dtype, K):
    """Entries whose quotient lies on a border (k + 1/2) or one step of the type beside it."""
    odd = torch.arange(K, device=DEV) % 127 * 2 + 1
    rows = []
    for top in (254.0, 127.0, 63.5):
        x = (odd * top / 254).to(dtype)            # 127 x / top = odd / 2, exact in every type
        x[::2] = -x[::2]
        x[K - 1] = top
        step = torch.finfo(dtype).eps
        up, down = x.float() * (1 + step), x.float() * (1 - step)
        for v in (x.float(), up, down):
            v = v.clamp(-top, top)
            rows.append(v.to(dtype))
    x = torch.stack(rows)
    q, scale, values = lq.quant_i8(x, values=True)
    check_exact(x, q, scale, values)


def test_quant_random_borders_fp32():
    """fp32 entries rounded from exact border quotients of random row maxima."""
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.rand(64, 1, generator=g, device=DEV, dtype=torch.float64) + 0.5
    a = a.float().double()
    k = torch.randint(-127, 127, (64, 1000), generator=g, device=DEV).double()
    x = ((k + 0.5) * a / 127).float()
    x[:, 0] = a[:, 0].float()
    q, scale, values = lq.quant_i8(x, values=True)
    check_exact(x, q, scale, values)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quant_extreme_rows(dtype):
    x = rand(9, 96, F32, 3)
    x[0] = 0
    x[1] = -0.0
    x[2, 5] = float("inf")
    x[3, 0] = float("nan")
    x[4, 95] = float("-inf")
    x[5] = x[5] / x[5].abs().amax() * float(torch.finfo(dtype).max)
    x[6] *= torch.finfo(dtype).tiny
    x[7] = 0
    x[7, 11] = torch.finfo(dtype).smallest_normal / 4
    x[8] *= torch.finfo(dtype).tiny / 8
    x = x.to(dtype)
    q, scale, values = lq.quant_i8(x, values=True)
    check_exact(x, q, scale, values)


def test_quant_strides_and_alignment():
    base = rand(40, 2000, BF16, 9)
    for x in (base[:, :1024], base[:, 8:1032], base[:, 1:1025], base[::3, 16:528], base[:1, 3:60],
              base.view(80, 1000)[1::2, :992]):
        q, scale, values = lq.quant_i8(x, values=True)
        check_exact(x, q, scale, values)


def check_whitened(x, sign, chan, block):
    K = x.shape[1]
    q, scale, values = lq.quant_i8(x, sign=sign, chan_scale=chan, block=block, values=True)
    v, dv = ref.whiten(x, sign, chan, block)
    a = v.abs().amax(1)
    da = dv.amax(1)
    assert ((scale.double() - a / 127).abs() <= (da + 2 * ref.EPS32 * a) / 127).all()
    # the code is the rounding of a quotient whose entry and maximum are off by dv and da
    off = 127 * (dv + da[:, None]) / (a - da)[:, None] + 1e-12
    assert ((q[:, :K].double() - 127 * v / a[:, None]).abs() <= 0.5 + off).all()
    assert not q[:, K:].any()
    assert torch.equal(values, (q[:, :K].float() * scale[:, None]).to(x.dtype))


@pytest.mark.parametrize("rows", [2, 500])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("block", [4, 64, 256, 1024])
def test_quant_whitened_off_alignment(rows, dtype, block):
    """Rows that start off a 16-byte boundary, and signs and scales that do."""
    base = rand(rows, 2400, dtype, rows + block)
    sg, cs = signs(2050, 1), torch.rand(2050, device=DEV) + 0.5
    for x in (base[:, 1:1025], base[:, 3:2051], base[:, 8:1032]):
        K = x.shape[1]
        check_whitened(x, sg[1:K + 1], None, block)
        check_whitened(x, sg[1:K + 1].clone(), cs[1:K + 1], block)


@pytest.mark.parametrize("block,K", [(1, 24), (2, 30), (4, 100), (8, 8), (16, 48), (32, 32),
                                     (64, 320), (128, 1152), (256, 256), (256, 8192),
                                     (256, 28672), (512, 1536), (1024, 5120), (2048, 2048),
                                     (4096, 12288), (4096, 53248)])
@pytest.mark.parametrize("rows,dtype", [(1, F32), (3, BF16), (310, F16)])
def test_quant_whitened(block, K, rows, dtype):
    x = rand(rows, K, dtype, K + block)
    x[0, 1] = 30.0
    cs = torch.rand(K, device=DEV) + 0.5
    for sign, chan in ((signs(K, 2), None), (signs(K, 3), cs), (None, None)):
        check_whitened(x, sign, chan, block)


def test_quant_outputs_stay_inside():
    """Nothing is written behind the last row of any output."""
    rows, K = 5, 100
    x = rand(rows, K, F16, 1)
    q = torch.full((rows + 2, 112), 99, dtype=torch.int8, device=DEV)
    scale = torch.full((rows + 3,), 7.0, device=DEV)
    values = torch.full((rows + 2, K), 5.0, dtype=F16, device=DEV)
    rc = lq.lib().lq_quant_i8(x.data_ptr(), lq.LQ_F16, rows, K, K, None, q.data_ptr(),
                              scale.data_ptr(), values.data_ptr(),
                              torch.cuda.current_stream().cuda_stream)
    assert rc == lq.LQ_OK
    check_exact(x, q[:rows], scale[:rows], values[:rows])
    assert (q[rows:] == 99).all() and (scale[rows:] == 7).all() and (values[rows:] == 5).all()


# ------------------------------------------------------------------ the product


def int8(rows, K, seed, lo=-127, fill=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.full((rows, lq.i8_row_bytes(K)), fill, dtype=torch.int8, device=DEV)
    q[:, :K] = torch.randint(lo, 128, (rows, K), generator=g, device=DEV).to(torch.int8)
    return q


def scales(n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.rand(n, generator=g, device=DEV) * 0.02 + 1e-3


def check_gemm(batch, K, N, dtype, bias, route=None, fill=0, lo=-127, ws=None):
    xq, wq = int8(batch, K, 1, lo, fill), int8(N, K, 2, lo, fill)
    xs, sw = scales(batch, 3), scales(N, 4)
    b = torch.randn(N, device=DEV) if bias else None
    ws = lq.new_i8_workspace() if ws is None else ws
    pad = torch.full((batch + 2, N), -3.0, dtype=dtype, device=DEV)
    y = lq.gemm_i8(xq, xs, wq, sw, K=K, bias=b, y=pad[:batch], workspace=ws, route=route)
    assert lq.device_status(ws) == (lq.LQ_OK, 0)
    ref.within(y, *ref.product(xq, xs, wq, sw, K, b))
    assert (pad[batch:] == -3).all()


SHAPES = [(1, 1, 1), (1, 16, 16), (1, 4096, 300), (2, 100, 33), (7, 4100, 1003), (8, 257, 129),
          (9, 512, 17), (16, 1000, 260), (17, 640, 128), (32, 8192, 200), (33, 128, 40),
          (64, 96, 500), (65, 300, 129), (128, 2048, 256), (129, 64, 1), (200, 1000, 777),
          (256, 160, 384), (300, 4096, 1000), (513, 250, 1030), (260, 1024, 10000),
          (1100, 384, 4104), (2049, 256, 1000), (700, 130, 5001), (1024, 2048, 8190)]


@pytest.mark.parametrize("batch,K,N", SHAPES)
def test_gemm(batch, K, N):
    for dtype, bias in ((F32, False), (BF16, True), (F16, False)):
        check_gemm(batch, K, N, dtype, bias)


@pytest.mark.parametrize("batch,K,N", [(1, 4096, 300), (5, 333, 70), (16, 1000, 260),
                                       (8, 8192, 200), (13, 17, 1), (9, 130, 33)])
@pytest.mark.parametrize("route", [lq.I8_ROUTE_GEMV, lq.I8_ROUTE_TC])
def test_gemm_small_batches_on_both_routes(batch, K, N, route):
    check_gemm(batch, K, N, F32, True, route=route)


@pytest.mark.parametrize("batch,K,N", [(1, 1, 1), (3, 128, 256), (17, 100, 257), (31, 8192, 8),
                                       (33, 2048, 1000), (64, 4100, 515), (100, 128, 30),
                                       (129, 1000, 2050), (256, 512, 512), (257, 384, 770),
                                       (700, 640, 5001), (1025, 200, 300), (300, 2056, 19000)])
@pytest.mark.parametrize("route", [lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR, lq.I8_ROUTE_SPLIT])
def test_gemm_tile_kernels(batch, K, N, route):
    check_gemm(batch, K, N, BF16, False, route=route)
    check_gemm(batch, K, N, F32, True, route=route)


@pytest.mark.parametrize("batch,K,N", [(1, 14337, 64), (9, 15000, 130), (16, 20480, 1184),
                                       (20, 8192, 1024), (40, 131071, 64), (85, 6912, 238),
                                       (404, 5000, 441), (1000, 2048, 256), (19, 16752, 5218)])
def test_gemm_by_clusters_along_k(batch, K, N):
    """Layers of few tiles, which the library's own choice splits along K."""
    assert lq.gemm_i8_route(batch, K, N) == lq.I8_ROUTE_SPLIT
    for dtype in (BF16, F16, F32):
        check_gemm(batch, K, N, dtype, dtype != F16)


@pytest.mark.parametrize("route", [lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR, lq.I8_ROUTE_SPLIT])
def test_gemm_tiles_with_odd_rows_of_y(route):
    """16-bit outputs at an odd width or off a 4-byte boundary are stored one by one."""
    check_gemm(70, 256, 333, F16, True, route=route)
    batch, K, N = 70, 256, 334
    xq, wq, xs, sw = int8(batch, K, 1), int8(N, K, 2), scales(batch, 3), scales(N, 4)
    flat = torch.zeros(batch * N + 1, dtype=BF16, device=DEV)
    y = lq.gemm_i8(xq, xs, wq, sw, y=flat[1:].view(batch, N), route=route)
    ref.within(y, *ref.product(xq, xs, wq, sw, K, None))
    assert flat[0] == 0


@pytest.mark.parametrize("batch", [3, 40, 300])
def test_gemm_ignores_the_padding(batch):
    check_gemm(batch, 1003, 150, F32, False, fill=77)


@pytest.mark.parametrize("batch", [2, 20, 70])
def test_gemm_longest_sums(batch):
    """The largest magnitudes of the longest rows: sums next to 2^31, both signs."""
    K, N = 131071, 48
    xq, wq = int8(batch, K, 1), int8(N, K, 2)
    xq[0, :K], wq[0, :K] = -128, -128
    xq[1, :K], wq[1, :K] = 127, 127
    one = torch.ones(batch, device=DEV)
    y = lq.gemm_i8(xq, one, wq, torch.ones(N, device=DEV), K=K)
    assert y[0, 0].item() == float(torch.tensor(128 * 128 * K, dtype=F32))
    ref.within(y, *ref.product(xq, one, wq, torch.ones(N, device=DEV), K, None))


@pytest.mark.parametrize("batch", [4, 30, 130])
def test_gemm_entries_of_minus_128_and_bad_scales(batch):
    check_gemm(batch, 500, 64, F32, True, lo=-128)
    K, N = 64, 32
    xq, wq, xs, sw = int8(batch, K, 1), int8(N, K, 2), scales(batch, 3), scales(N, 4)
    xs[1] = float("nan")
    y = lq.gemm_i8(xq, xs, wq, sw)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


def test_gemm_full_size_layers():
    for batch, K, N in ((1, 8192, 28672), (16, 28672, 8192), (2048, 8192, 28672)):
        check_gemm(batch, K, N, BF16, False)


def test_offsets_past_32_bits():
    """Rows whose elements lie beyond 2^31 equal the same rows on their own."""
    rows, K = 270000, 8192
    x = torch.empty(rows, K, dtype=BF16, device=DEV)
    x[:] = rand(1000, K, BF16, 1).repeat(rows // 1000, 1)
    x[-1] = rand(1, K, BF16, 2)
    q, s = lq.quant_i8(x, block=256)
    for at in (0, rows // 2, rows - 3):
        q2, s2 = lq.quant_i8(x[at:at + 3].clone(), block=256)
        assert torch.equal(q[at:at + 3], q2) and torch.equal(s[at:at + 3], s2)
    del q, s
    pre = lq.Norm("rms")
    c, n = lq.norm_residual(x, x, None, pre)
    c2, n2 = lq.norm_residual(x[-3:].clone(), x[-3:].clone(), None, pre)
    # the two calls split a row over threads differently: one rounding step of bf16 apart at most
    assert torch.equal(c[-3:], c2)
    assert ((n[-3:].float() - n2.float()).abs() <= 2.0 ** -7 * n2.float().abs()).all()
    del x, c, n
    batch, K, N = 70000, 64, 32768
    xq, wq, xs, sw = int8(batch, K, 1), int8(N, K, 2), scales(batch, 3), scales(N, 4)
    for route in (lq.I8_ROUTE_TC, lq.I8_ROUTE_PAIR, lq.I8_ROUTE_SPLIT):
        y = lq.gemm_i8(xq, xs, wq, sw, dtype=BF16, route=route)
        ref.within(y[-5:], *ref.product(xq[-5:], xs[-5:], wq, sw, K, None))
        ref.within(y[:5], *ref.product(xq[:5], xs[:5], wq, sw, K, None))
        del y


def test_gemm_empty():
    wq, sw = int8(10, 64, 1), scales(10, 1)
    y = lq.gemm_i8(int8(0, 64, 1), scales(0, 1), wq, sw)
    assert y.shape == (0, 10)
    y = lq.gemm_i8(int8(3, 64, 1), scales(3, 1), wq[:0], sw[:0])
    assert y.shape == (3, 0)
    q, s = lq.quant_i8(torch.empty(0, 40, device=DEV))
    assert q.shape == (0, 48) and s.shape == (0,)


def test_gemm_same_bits_every_time():
    for batch in (3, 40, 300):
        xq, wq, xs, sw = int8(batch, 4096, 1), int8(1000, 4096, 2), scales(batch, 3), scales(1000, 4)
        y = lq.gemm_i8(xq, xs, wq, sw)
        assert torch.equal(y, lq.gemm_i8(xq, xs, wq, sw))
        if batch <= 16:     # the integer sum does not depend on the kernel
            assert torch.equal(y, lq.gemm_i8(xq, xs, wq, sw, route=lq.I8_ROUTE_TC))
        assert torch.equal(y, lq.gemm_i8(xq, xs, wq, sw, route=lq.I8_ROUTE_PAIR))
        assert torch.equal(y, lq.gemm_i8(xq, xs, wq, sw, route=lq.I8_ROUTE_SPLIT))


def test_graphs_share_a_workspace():
    """Two captured products share one workspace; each replay reads the inputs of its time."""
    ws = lq.new_i8_workspace()
    cases = []
    for batch, K, N in ((4, 1024, 500), (150, 2048, 300)):
        x = rand(batch, K, BF16, batch)
        wq, sw = int8(N, K, 2), scales(N, 3)

        def call(x=x, wq=wq, sw=sw):
            q, s = lq.quant_i8(x, block=256)
            return q, s, lq.gemm_i8(q, s, wq, sw, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        cases.append((x, wq, sw, g, out))
    for turn in range(3):
        for x, wq, sw, g, (q, s, y) in cases:
            x.copy_(rand(x.shape[0], x.shape[1], BF16, 50 + turn))
            g.replay()
        for x, wq, sw, g, (q, s, y) in cases:
            q2, s2 = lq.quant_i8(x, block=256)
            assert torch.equal(q, q2) and torch.equal(s, s2)
            ref.within(y, *ref.product(q, s, wq, sw, x.shape[1], None))
    assert lq.device_status(ws) == (lq.LQ_OK, 0)


def test_other_streams():
    side = torch.cuda.Stream()
    K, N = 2048, 600
    wq, sw = int8(N, K, 2), scales(N, 3)
    for batch in (2, 200):
        x = rand(batch, K, BF16, batch)
        side.wait_stream(torch.cuda.current_stream())
        q, s = lq.quant_i8(x, stream=side)
        y = lq.gemm_i8(q, s, wq, sw, stream=side)
        with torch.cuda.stream(side):
            y2 = lq.gemm_i8(q, s, wq, sw)
        side.synchronize()
        ref.within(y, *ref.product(q, s, wq, sw, K, None))
        assert torch.equal(y, y2)


def test_call_while_another_device_is_current(monkeypatch):
    """With another device current, a call makes its tensors' device current and runs there."""
    entered = []
    real = torch.cuda.device

    class Spy(real):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

    x = rand(3, 256, BF16, 1)
    wq, sw = int8(8, 256, 1), scales(8, 1)
    q, s = lq.quant_i8(x)
    y = lq.gemm_i8(q, s, wq, sw)
    r, n = lq.norm_residual(x, x, None, lq.Norm("rms"))
    monkeypatch.setattr(torch.cuda, "device", Spy)

    def elsewhere():
        answers = iter((torch.cuda.current_device() + 1, torch.cuda.current_device()))
        monkeypatch.setattr(lq, "_current_device", lambda: next(answers))

    elsewhere()
    q2, s2 = lq.quant_i8(x)
    elsewhere()
    y2 = lq.gemm_i8(q, s, wq, sw)
    elsewhere()
    r2, n2 = lq.norm_residual(x, x, None, lq.Norm("rms"))
    assert entered == [x.get_device()] * 3
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(y, y2)
    assert torch.equal(r, r2) and torch.equal(n, n2)


def test_refused_tensors():
    x = rand(4, 64, BF16, 1)
    q, s = lq.quant_i8(x)
    wq, sw = int8(8, 64, 1), scales(8, 1)
    with pytest.raises(TypeError, match="CUDA tensor"):
        lq.gemm_i8(q, s, wq.cpu(), sw)
    with pytest.raises(TypeError, match="dtype"):
        lq.gemm_i8(q, s.double(), wq, sw)
    with pytest.raises(ValueError, match="shape"):
        lq.gemm_i8(q, s[:3], wq, sw)
    with pytest.raises(ValueError, match="shape"):
        lq.gemm_i8(q, s, wq[:, :48].contiguous(), sw)
    with pytest.raises(ValueError, match="contiguous"):
        lq.gemm_i8(q, s, int8(8, 128, 1)[:, :64], sw)
    with pytest.raises(ValueError, match="bytes"):
        lq.gemm_i8(q, s, wq, sw, K=65)
    with pytest.raises(lq.LQError, match="GEMV route"):
        lq.gemm_i8(int8(17, 64, 1), scales(17, 1), wq, sw, route=lq.I8_ROUTE_GEMV)
    with pytest.raises(TypeError, match="dtype"):
        lq.quant_i8(x.double())
    with pytest.raises(ValueError, match="dense rows"):
        lq.quant_i8(x.t())
    with pytest.raises(ValueError, match="dense rows"):
        lq.quant_i8(x[:1].expand(4, 64))
    with pytest.raises(lq.LQError, match="divide"):
        lq.quant_i8(x, block=128)
    with pytest.raises(ValueError, match="shape"):
        lq.quant_i8(x, sign=signs(63, 1), block=64)
    assert ctypes.sizeof(lq.NormDesc) == 32
