"""lq_norm_residual against its formula in 64 bits, and a block's run through the operators."""
import pytest
import torch

import fractional_bit_weight_b200 as lq
from fractional_bit_weight_b200 import synth
from gpu_helpers import assert_close, device_layer, oracle_rows
import w8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(shape, dtype, g, scale=1.0, shift=0.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV) + shift).to(dtype)


def make_norm(kind, K, dtype, g, bias, eps=1e-5, weight=True):
    if kind is None:
        return None, None
    w = rand((K,), dtype, g, 0.2, 1.0) if weight else None
    b = rand((K,), dtype, g, 0.3) if bias else None
    return lq.Norm(kind, w, b, eps), (kind, w, b, eps)


def gate_rows(gate, rows, tokens):
    t = torch.arange(rows, device=DEV) // tokens
    return gate.reshape(-1, gate.shape[-1])[t]


def check(rows, K, hdt, rdt, ndt, post, pre, gate=None, seed=0, branch=0.7, resid=1.1, bias=False,
          shift=0.0, norm_dt=None):
    g = gen(seed + rows * 31 + K)
    h = rand((rows, K), hdt, g, 2.0, shift)
    r = None if rdt is None else rand((rows, K), rdt, g, 3.0, shift)
    ndt_w = norm_dt or hdt
    post, post_ref = make_norm(post, K, ndt_w, g, bias)
    pre, pre_ref = make_norm(pre, K, ndt_w, g, bias)
    gt, tokens, rows_ref = None, 0, None
    if gate is not None:
        tokens, cols = gate
        gt = rand((-(-rows // tokens), cols), rdt or hdt, g, 0.5, 0.5)
        rows_ref = gate_rows(gt, rows, tokens)
    c, n = lq.norm_residual(h, r, post, pre, gt, tokens, branch, resid, dtype=ndt)
    wc, dc, wn, dn = ref.boundary(h, r, post_ref, pre_ref, rows_ref, branch, resid)
    assert n.dtype == ndt
    ref.within(n, wn, dn)
    if r is None:
        assert c is None
    else:
        assert c.dtype == rdt
        ref.within(c, wc, dc)
    # as int8: the codes of what n is before its rounding
    c2, q, s, n2 = lq.norm_residual_i8(h, r, post, pre, gt, tokens, branch, resid, dtype=F32)
    if r is not None:
        assert torch.equal(c, c2)
    ref.within(n2, wn, dn)
    q3, s3 = lq.quant_i8(n2)
    assert torch.equal(q, q3) and torch.equal(s, s3)
    if ndt == F32:
        assert torch.equal(n, n2)


SIZES = [(1, 1), (1, 8), (2, 7), (1, 8192), (3, 1000), (5, 4097), (297, 256), (300, 8192),
         (310, 1001), (2, 16384), (1, 28672), (2, 20001), (1, 40000), (1, 65536)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_sandwich(rows, K, kind):
    check(rows, K, F32, BF16, BF16, kind, kind, bias=kind == "layer")


@pytest.mark.parametrize("hdt", [F32, F16, BF16])
@pytest.mark.parametrize("rdt", [F32, F16, BF16, None])
@pytest.mark.parametrize("ndt", [F32, F16, BF16])
def test_types(hdt, rdt, ndt):
    check(5, 520, hdt, rdt, ndt, "rms", "layer", gate=(2, 520), bias=True)
    check(3, 333, hdt, rdt, ndt, "layer", "rms", gate=(1, 1))
    check(300, 2048, hdt, rdt, ndt, "rms", "rms", norm_dt=F32)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", [None, (1, 1), (1, 264), (4, 264), (100, 264), (100, 1)])
def test_parts(post, pre, gate):
    check(11, 264, BF16, F32, F32, post, pre, gate, branch=-0.3, resid=0.5)


def test_rows_far_from_zero():
    """A mean far larger than the spread: the variance comes from the centred values."""
    check(4, 3000, F32, F32, F32, "layer", "layer", shift=1000.0, bias=True)
    check(4, 2048, F32, F32, F32, "layer", "rms", shift=-300.0)


def test_degenerate_rows():
    K = 96
    h = torch.zeros(6, K, device=DEV)
    h[1] = 5.0                    # no variance
    h[2, 0] = float("inf")
    h[3, 7] = float("nan")
    h[4] = 1e-30
    h[5] = 1e18                   # the squares' sum still fits fp32
    r = torch.ones(6, K, device=DEV)
    c, n = lq.norm_residual(h, r, lq.Norm("layer", eps=1e-5), lq.Norm("rms", eps=1e-5))
    ok = [0, 1, 4, 5]
    wc, dc, wn, dn = ref.boundary(h[ok], r[ok], ("layer", None, None, 1e-5),
                                  ("rms", None, None, 1e-5), None, 1.0, 1.0)
    ref.within(c[ok], wc, dc)
    ref.within(n[ok], wn, dn)
    assert torch.isnan(c[3]).all() and torch.isnan(n[3]).all() and torch.isnan(c[2]).any()
    # an infinite or NaN row has no codes and a NaN scale; the others are not touched by it
    _, q, s = lq.norm_residual_i8(h, r, lq.Norm("layer", eps=1e-5), lq.Norm("rms", eps=1e-5))
    assert torch.isnan(s[[2, 3]]).all() and not q[[2, 3]].any() and torch.isfinite(s[ok]).all()
    # eps = 0 and a zero row is 0 / 0
    _, n = lq.norm_residual(h[:1], None, None, lq.Norm("rms", eps=0.0))
    assert torch.isnan(n).all()


@pytest.mark.parametrize("rows,block,K", [(1, 256, 8192), (3, 4, 100), (301, 256, 1024),
                                          (2, 1024, 5120), (2, 4096, 8192)])
def test_whitened_codes(rows, block, K):
    g = gen(K)
    h, r = rand((rows, K), F32, g), rand((rows, K), BF16, g)
    sign = torch.randint(0, 2, (K,), generator=g, device=DEV).to(torch.int8) * 2 - 1
    pre = lq.Norm("rms", rand((K,), BF16, g, 0.2, 1.0))
    _, q, s, n = lq.norm_residual_i8(h, r, None, pre, sign=sign, block=block, dtype=F32)
    q2, s2 = lq.quant_i8(n, sign=sign, block=block)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("K", [512, 500, 501])
def test_in_place_and_strides(K):
    g = gen(K)
    big = rand((9, 1200), BF16, g)
    h = rand((9, 700), F32, g)[:, 4:4 + K]
    pre = lq.Norm("rms", None, None, 1e-5)
    want_c, want_n = lq.norm_residual(h.contiguous(), big[:, 8:8 + K].contiguous(), None, pre)
    r = big.clone()
    view = r[:, 8:8 + K]
    c, n = lq.norm_residual(h, view, None, pre, residual_out=view)
    assert c is view and torch.equal(view, want_c) and torch.equal(n, want_n)
    assert torch.equal(r[:, :8], big[:, :8]) and torch.equal(r[:, 8 + K:], big[:, 8 + K:])
    out = torch.full((11, K), 2.0, dtype=BF16, device=DEV)
    c, n = lq.norm_residual(h, big[:, 8:8 + K], None, pre, residual_out=out[:9])
    assert torch.equal(out[:9], want_c) and (out[9:] == 2).all()
    # without a residual, c is the scaled branch
    c, n = lq.norm_residual(h, None, None, None, branch_scale=0.5, residual_out=out[:9], dtype=F32)
    assert torch.equal(n, h * 0.5) and torch.equal(c, (h * 0.5).to(BF16))


@pytest.mark.parametrize("rows,K", [(3, 100), (3, 4096), (600, 1000), (600, 2048), (2, 20000),
                                    (300, 9001)])
def test_outputs_stay_inside(rows, K):
    """Nothing is written before or behind any output."""
    g = gen(K)
    h, r = rand((rows, K), F32, g), rand((rows, K), BF16, g)
    ks = lq.i8_row_bytes(K)

    def guarded(shape, dtype, fill):
        n = 1
        for d in shape:
            n *= d
        flat = torch.full((n + 256,), fill, dtype=dtype, device=DEV)
        return flat, flat[128:128 + n].view(shape)

    bufs = [guarded((rows, K), BF16, 3.0), guarded((rows, K), F16, 4.0),
            guarded((rows, ks), torch.int8, 55), guarded((rows,), F32, 6.0)]
    c, n, q, s = (v for _, v in bufs)
    pre = lq.Norm("layer", None, None, 1e-5)
    rc = lq.lib().lq_norm_residual(
        h.data_ptr(), lq.LQ_F32, K, r.data_ptr(), lq.LQ_BF16, K, rows, K, pre._ref, None, 1.0, 1.0,
        c.data_ptr(), pre._ref, n.data_ptr(), lq.LQ_F16, None, q.data_ptr(), s.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    assert rc == lq.LQ_OK
    for (flat, _), fill in zip(bufs, (3.0, 4.0, 55, 6.0)):
        assert (flat[:128] == fill).all() and (flat[-128:] == fill).all()
    c2, q2, s2, n2 = lq.norm_residual_i8(h, r, pre, pre, dtype=F16)
    for got, want in ((c, c2), (n, n2), (q, q2), (s, s2)):
        assert torch.equal(got, want)


def test_weights_off_alignment():
    K = 512
    g = gen(1)
    h = rand((4, K), BF16, g)
    w = rand((K + 1,), BF16, g)
    a = lq.norm_residual(h, None, None, lq.Norm("rms", w[1:]))[1]
    b = lq.norm_residual(h, None, None, lq.Norm("rms", w[1:].clone()))[1]
    ref.within(a, *ref.boundary(h, None, None, ("rms", w[1:], None, 1e-6), None, 1., 1.)[2:])
    ref.within(b, *ref.boundary(h, None, None, ("rms", w[1:], None, 1e-6), None, 1., 1.)[2:])


def test_refusals():
    g = gen(2)
    h, r = rand((4, 64), F32, g), rand((4, 64), BF16, g)
    with pytest.raises(ValueError, match="norm kind"):
        lq.Norm("batch")
    with pytest.raises(TypeError, match="one dtype"):
        lq.Norm("rms", torch.ones(64, device=DEV), torch.ones(64, device=DEV, dtype=BF16))
    with pytest.raises(ValueError, match="norm over 63"):
        lq.norm_residual(h, r, lq.Norm("rms", torch.ones(63, device=DEV)))
    with pytest.raises(TypeError, match="Norm objects"):
        lq.norm_residual(h, r, torch.ones(64, device=DEV))
    with pytest.raises(ValueError, match="shape"):
        lq.norm_residual(h, r[:, :63])
    with pytest.raises(ValueError, match="gate"):
        lq.norm_residual(h, r, gate=torch.ones(3, 64, device=DEV), gate_tokens=2)
    with pytest.raises(lq.LQError, match="gate cols"):
        lq.norm_residual(h, r, gate=torch.ones(4, 63, device=DEV))
    with pytest.raises(lq.LQError, match="eps"):
        lq.norm_residual(h, r, lq.Norm("rms", eps=-1.0))
    with pytest.raises(TypeError, match="CUDA tensor"):
        lq.norm_residual(h.cpu(), r)
    with pytest.raises(TypeError, match="residual_out has dtype"):
        lq.norm_residual(h, r, residual_out=torch.empty(4, 64, device=DEV))
    assert lq.norm_residual(h[:0], r[:0], lq.Norm("rms"), lq.Norm("rms"))[1].shape == (0, 64)


def test_capture_and_side_stream():
    g = gen(3)
    h, r = rand((5, 2048), F32, g), rand((5, 2048), BF16, g)
    pre = lq.Norm("rms", rand((2048,), BF16, g, 0.2, 1.0))
    want = lq.norm_residual(h, r, pre, pre)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lq.norm_residual(h, r, pre, pre)
    for _ in range(2):
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    h.copy_(rand((5, 2048), F32, g))
    graph.replay()
    want = lq.norm_residual(h, r, pre, pre)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lq.norm_residual(h, r, pre, pre, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("batch", [1, 7, 70])
def test_block_of_8_bit_and_fractional_layers(orc, batch):
    """The operators as a block uses them: boundary into int8 rows, an 8-bit projection, a second
    boundary into a float row, and the fractional-bit layer on it. Each stage is held to its
    definition on the inputs it got."""
    K, mid, d, D = 1024, 1280, 10, 24
    g = gen(batch)
    h, r = rand((batch, K), F32, g, 2.0), rand((batch, K), BF16, g, 3.0)
    sign = torch.randint(0, 2, (K,), generator=g, device=DEV).to(torch.int8) * 2 - 1
    norms = [make_norm("rms", K, BF16, g, False) for _ in range(2)]
    w = rand((mid, K), F32, g, K ** -0.5)
    wq, sw = lq.quant_i8(w, sign=sign, block=256)     # H is orthogonal: (W T^t)(T x) = W x
    ws = lq.new_i8_workspace()

    c, q, s, n = lq.norm_residual_i8(h, r, norms[0][0], norms[1][0], sign=sign, block=256,
                                     dtype=F32)
    wc, dc, wn, dn = ref.boundary(h, r, norms[0][1], norms[1][1], None, 1.0, 1.0)
    ref.within(c, wc, dc)
    ref.within(n, wn, dn)
    y = lq.gemm_i8(q, s, wq, sw, workspace=ws)
    ref.within(y, *ref.product(q, s, wq, sw, K, None))
    # against the layer in full precision: 8-bit noise of both operands (each about a third of
    # amax / 127 per entry, amax about 4 sigma) is near 1.3 % of y; 4 % is far outside it
    full = n.double() @ w.double().t()
    assert (y.double() - full).norm() <= 0.04 * full.norm()
    assert lq.device_status(ws) == (lq.LQ_OK, 0)

    r2 = rand((batch, mid), BF16, g, 3.0)
    pre = make_norm("rms", mid, BF16, g, False)
    c2, x2 = lq.norm_residual(y, r2, None, pre[0], dtype=BF16)
    wc, dc, wn, dn = ref.boundary(y, r2, None, pre[1], None, 1.0, 1.0)
    ref.within(c2, wc, dc)
    ref.within(x2, wn, dn)
    layer = synth.make_layer("block", 5, 1, mid, 200, d, D, batch)
    dl = device_layer(layer)
    out = lq.gemm(x2, dl["packed"], dl["M"], dl["s"], d, D, sign=dl["sign"], block=layer.block)
    layer.x = x2.float().cpu().numpy()
    import numpy as np
    assert_close(out.cpu().numpy(), oracle_rows(orc, layer, np.arange(200)),
                 f"block of both kinds, batch {batch}")


@pytest.mark.parametrize("batch,K", [(1, 2048), (5, 8192), (3, 12288), (40, 1024), (300, 2048)])
def test_back_to_back_equals_one_at_a_time(batch, K):
    """A chain whose calls read what the ones before wrote, in place and into reused memory: run
    without a pause, replayed as a graph, and with a wait after every call, all bits agree."""
    g = gen(batch + K)
    h0, r0 = rand((batch, K), F32, g, 2.0), rand((batch, K), BF16, g, 3.0)
    pre = lq.Norm("rms", rand((K,), BF16, g, 0.2, 1.0), None, 1e-5)
    wq, sw = lq.quant_i8(rand((K, K), BF16, g, K ** -0.5))
    ws = lq.new_i8_workspace()

    def chain(h, r, pause):
        for _ in range(6):
            r, q, s = lq.norm_residual_i8(h, r, pre, pre, residual_out=r, branch_scale=0.5,
                                          block=256)
            pause()
            h = lq.gemm_i8(q, s, wq, sw, workspace=ws)
            pause()
            r, n = lq.norm_residual(h, r, None, pre, residual_out=r, dtype=F32)
            pause()
            q, s = lq.quant_i8(n, block=256)
            pause()
            h = lq.gemm_i8(q, s, wq, sw, workspace=ws)
            pause()
        return h, r

    want = chain(h0, r0.clone(), torch.cuda.synchronize)
    for _ in range(3):
        got = chain(h0, r0.clone(), lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    r1 = r0.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(h0, r1, lambda: None)
    for _ in range(3):
        r1.copy_(r0)
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert lq.device_status(ws) == (lq.LQ_OK, 0)


def test_two_streams_at_once():
    """Independent chains on two streams, one workspace for both: nothing but the status is shared."""
    g = gen(4)
    K, N = 4096, 4096
    w = [lq.quant_i8(rand((N, K), BF16, g, K ** -0.5)) for _ in range(2)]
    xs = [rand((b, K), BF16, g) for b in (6, 200)]
    ws = lq.new_i8_workspace()

    def run(i):
        x = xs[i]
        for _ in range(8):
            q, s = lq.quant_i8(x, block=256)
            x = lq.gemm_i8(q, s, *w[i], dtype=BF16, workspace=ws)
        return x

    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(run(i))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert lq.device_status(ws) == (lq.LQ_OK, 0)
