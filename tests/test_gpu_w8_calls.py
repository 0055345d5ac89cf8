"""Calls of the 8-bit and boundary operators that the other tests do not make."""
import os
import subprocess
import sys

import pytest
import torch

import fractional_bit_weight_b200 as lq
import w8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(shape, dtype, g, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def test_norms_follow_their_tensors():
    """A module that changes its type or is loaded anew keeps its Parameter objects."""
    g = gen(1)
    h = rand((5, 520), F32, g)
    module = torch.nn.LayerNorm(520, device=DEV)
    norm = lq.Norm("layer", module.weight, module.bias, 1e-5)
    for dtype in (F32, BF16, F16, F32):
        module.to(dtype)
        for t in (module.weight, module.bias):
            t.data = rand((520,), dtype, g)
        got = lq.norm_residual(h, None, norm, norm, dtype=F32)[1]
        fresh = lq.Norm("layer", module.weight, module.bias, 1e-5)
        assert torch.equal(got, lq.norm_residual(h, None, fresh, fresh, dtype=F32)[1])
        stats = ("layer", module.weight.detach(), module.bias.detach(), 1e-5)
        ref.within(got, *ref.boundary(h, None, stats, stats, None, 1.0, 1.0)[2:])


def test_boundary_of_an_empty_batch():
    h = torch.empty(0, 64, device=DEV)
    for gate, tokens in ((torch.empty(0, 64, device=DEV), 0), (torch.empty(0, 1, device=DEV), 5),
                         (torch.ones(64, device=DEV), 0)):
        c, n = lq.norm_residual(h, h, None, lq.Norm("rms"), gate, tokens)
        assert c.shape == n.shape == (0, 64)
        c, q, s = lq.norm_residual_i8(h, h, None, None, gate, tokens, block=64)
        assert q.shape == (0, 64) and s.shape == (0,)


def test_boundary_in_place_over_its_input():
    """c may take the place of h as it may that of the residual."""
    g = gen(2)
    for rows, K in ((3, 1000), (400, 1000), (2, 20000), (5, 333)):
        pre = lq.Norm("rms", rand((K,), F32, g))
        h, r = rand((rows, K), BF16, g), rand((rows, K), BF16, g)
        want = lq.norm_residual(h, r, pre, pre)
        for args, out in (((h.clone(), r), 0), ((h, r.clone()), 1)):
            c, n = lq.norm_residual(*args, pre, pre, residual_out=args[out])
            assert c is args[out] and torch.equal(c, want[0]) and torch.equal(n, want[1])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,K", [(3, 264), (300, 2048), (2, 333), (300, 1001), (2, 20000)])
def test_channel_scales_without_rotation(rows, K, dtype):
    """block = 1: the codes of sign . chan_scale . x. The scales are powers of two, so that the
    products are exact and the codes those of the definition."""
    g = gen(K)
    x = rand((rows, K), dtype, g)
    scale = torch.exp2(torch.randint(-3, 4, (K,), generator=g, device=DEV).float())
    sign = torch.randint(0, 2, (K,), generator=g, device=DEV).to(torch.int8) * 2 - 1
    for sg, cs in ((sign, None), (None, scale), (sign, scale)):
        q, s, v = lq.quant_i8(x, sign=sg, chan_scale=cs, block=1, values=True)
        t = x.double() * (1 if sg is None else sg.double()) * (1 if cs is None else cs.double())
        want, ws = ref.codes(t)
        off = 127 * (q[:, :K].double() / 127 - t / t.abs().amax(1, keepdim=True))
        # half to even from an approximate quotient: a code next to a border may fall either way
        assert (off.abs() <= 0.5 + 127 * 2 * ref.EPS32).all() and not q[:, K:].any()
        assert ((s.double() - ws).abs() <= 2 * ref.EPS32 * ws).all()
        assert torch.equal(v, (q[:, :K].float() * s[:, None]).to(dtype))
        _, q2, s2, n = lq.norm_residual_i8(x, sign=sg, chan_scale=cs, block=1, dtype=F32)
        assert torch.equal(n, x.float()) and torch.equal(s, s2)
        assert int((q != q2).sum()) <= int((off.abs() > 0.5 - 127 * 2 * ref.EPS32).sum())


def test_status_of_calls_without_a_workspace():
    g = gen(3)
    q, s = lq.quant_i8(rand((40, 256), BF16, g))
    wq, sw = lq.quant_i8(rand((100, 256), BF16, g))
    y = lq.gemm_i8(q, s, wq, sw)
    ws = lq.default_i8_workspace()
    assert lq.device_status(ws) == (lq.LQ_OK, 0)
    # a bounded wait that runs out records itself there; the next product is right
    lq.check_wait_timeout(ws, 5)
    assert lq.device_status(ws) == (lq.LQ_ETIMEOUT, lq.LQ_ETIMEOUT)
    assert torch.equal(y, lq.gemm_i8(q, s, wq, sw)) and lq.device_status(ws) == (lq.LQ_OK, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = lq.gemm_i8(q, s, wq, sw, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and lq.default_i8_workspace("cuda:0") is ws
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lq.gemm_i8(q, s, wq, sw)
    out.zero_()
    graph.replay()
    assert torch.equal(out, y) and lq.default_i8_workspace() is ws


def test_first_call_captured(monkeypatch):
    """A call captured before any other makes its workspace part of the graph."""
    monkeypatch.setattr(lq, "_I8_WORKSPACES", {})
    g = gen(4)
    q, s = lq.quant_i8(rand((40, 256), BF16, g))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lq.gemm_i8(q, s, q, s)
    assert not lq._I8_WORKSPACES
    graph.replay()
    assert torch.equal(out, lq.gemm_i8(q, s, q, s))


def check_whitened(x, sign, chan, block, out):
    """Codes, scales and (or None) values of T(x) against 64 bits, as far as fp32 sums may be off."""
    q, scale, values = out
    K = x.shape[1]
    v, dv = ref.whiten(x, sign, chan, block)
    a, da = v.abs().amax(1), dv.amax(1)
    # the maximum's error, then its products with 1/sqrt(block) and 1/127
    assert ((scale.double() - a / 127).abs() <= (da + 2 * ref.EPS32 * a) / 127).all()
    off = 127 * (dv + da[:, None]) / (a - da)[:, None] + 1e-12
    assert ((q[:, :K].double() - 127 * v / a[:, None]).abs() <= 0.5 + off).all()
    assert not q[:, K:].any()
    if values is not None:
        assert torch.equal(values, (q[:, :K].float() * scale[:, None]).to(x.dtype))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("block,K", [(4, 36), (64, 320), (256, 1024), (256, 8192), (1024, 20480),
                                     (4096, 8192)])
@pytest.mark.parametrize("rows", [8, 520])
def test_largest_rows_under_rotation(rows, block, K, dtype):
    """Finite rows whose sums pass the largest fp32 before T's 1/sqrt(block), beside ordinary ones
    and ones that hold an infinity or a NaN."""
    g = gen(block + K)
    x = rand((rows, K), F32, g)
    sign = torch.randint(0, 2, (K,), generator=g, device=DEV).to(torch.int8) * 2 - 1
    top = torch.finfo(dtype).max
    for i in (0, 1):
        x[i::8] = (x[i::8] / x[i::8].abs().amax(1, keepdim=True)).double().mul(top).float()
    x[2::8] = top * sign.float()        # every sum of a block at its largest
    x[3::8] *= 2.0 ** 100 if dtype != F16 else 1.0
    x = x.to(dtype)
    x[4::8, K // 2] = float("inf")
    x[5::8, K - 1] = float("nan")
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[4::8] = bad[5::8] = True
    scale = torch.rand(K, generator=g, device=DEV) + 0.25
    for cs in (None, scale):
        out = lq.quant_i8(x, sign=sign, chan_scale=cs, block=block, values=True)
        q, s, v = out
        assert torch.isnan(s[bad]).all() and not q[bad].any() and torch.isnan(v[bad]).all()
        check_whitened(x[~bad], sign, cs, block, [t[~bad] for t in out])
        # rows off alignment, and the same rows as a branch without norms
        pad = torch.zeros(rows, K + 1, dtype=dtype, device=DEV)
        pad[:, 1:] = x
        for q2, s2 in (lq.quant_i8(pad[:, 1:], sign=sign, chan_scale=cs, block=block),
                       lq.norm_residual_i8(x, sign=sign, chan_scale=cs, block=block)[1:]):
            assert torch.isnan(s2[bad]).all() and not q2[bad].any()
            check_whitened(x[~bad], sign, cs, block, (q2[~bad], s2[~bad], None))


def test_scales_past_fp32_read_as_nan():
    """A channel scale may take T(x) / 127 past the largest fp32: such a row has no scale."""
    x = torch.full((2, 256), torch.finfo(F32).max, device=DEV)
    x[1] = 1.0
    cs = torch.full((256,), 2.0 ** 20, device=DEV)
    q, s, v = lq.quant_i8(x, chan_scale=cs, block=256, values=True)
    assert torch.isnan(s[0]) and not q[0].any() and torch.isnan(v[0]).all()
    check_whitened(x[1:], None, cs, 256, (q[1:], s[1:], v[1:]))


FIRST_CALLS_CAPTURED = """
import torch
import fractional_bit_weight_b200 as lq
x = torch.randn(40, 512, device="cuda")
w = torch.randn(300, 512, device="cuda")
wq = torch.zeros(300, 512, dtype=torch.int8, device="cuda")
ws = torch.zeros(300, device="cuda")
pre = lq.Norm("rms", torch.ones(512, device="cuda"))


def call():
    q, s = lq.quant_i8(w, block=256)
    wq.copy_(q)
    ws.copy_(s)
    c, q, s = lq.norm_residual_i8(x, x, None, pre, block=256)
    return [c, q, s] + [lq.gemm_i8(q[:n], s[:n], wq, ws, route=r)
                        for n, r in ((2, None), (40, None), (40, lq.I8_ROUTE_TC),
                                     (40, lq.I8_ROUTE_PAIR), (40, lq.I8_ROUTE_SPLIT))]


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(out, call()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_calls_of_a_process_captured():
    """The library looks the device up and raises its kernels' limits inside a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(lq.__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]
