"""What the binding of the 8-bit and boundary operators passes on, refuses and keeps. No GPU is
used: host and meta tensors stand in for the device's, and a recorder for the library."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import fractional_bit_weight_b200 as lq

HOST = -1                   # get_device() of a host or meta tensor
HUGE = 2 ** 32 + 4          # its low 32 bits are a small number


class Recorder:
    """Every entry point returns LQ_OK and leaves its arguments in calls."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(lq, "lib", lambda: r)
    monkeypatch.setattr(lq, "_device_of", lambda t, name: t.get_device())
    monkeypatch.setattr(lq, "_current_device", lambda: HOST)
    monkeypatch.setattr(lq, "_raw_stream", lambda device: 0)
    return r


def descriptor(call, kind):
    """The descriptor of this kind among a call's arguments."""
    return next(a._obj for a in call[1] if isinstance(getattr(a, "_obj", None), kind))


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_sizes_past_32_bits_are_refused(rec):
    i8 = torch.int8
    ws = torch.zeros(256, dtype=torch.uint8)
    calls = [lambda: lq.quant_i8(meta(HUGE, 1)), lambda: lq.quant_i8(meta(1, HUGE)),
             lambda: lq.norm_residual(meta(HUGE, 1)), lambda: lq.norm_residual_i8(meta(1, HUGE)),
             lambda: lq.gemm_i8(meta(HUGE, 16, dtype=i8), meta(HUGE), meta(4, 16, dtype=i8), meta(4),
                                workspace=ws),
             lambda: lq.gemm_i8(meta(4, 16, dtype=i8), meta(4), meta(HUGE, 16, dtype=i8), meta(HUGE),
                                workspace=ws),
             lambda: lq.gemm_i8(meta(1, 2 ** 32 + 16, dtype=i8), meta(1),
                                meta(1, 2 ** 32 + 16, dtype=i8), meta(1), workspace=ws),
             lambda: lq.gemm_i8(meta(4, 16, dtype=i8), meta(4), meta(4, 16, dtype=i8), meta(4),
                                workspace=ws, route=2 ** 32),
             lambda: lq.quant_i8(meta(4, 512), block=2 ** 32 + 256),
             lambda: lq.norm_residual(meta(4, 64), gate=meta(1, 2 ** 32 + 64)),
             lambda: lq.i8_row_bytes(HUGE), lambda: lq.gemm_i8_route(HUGE, 64, 64),
             lambda: lq.gemm_i8_plan(4, HUGE, 64), lambda: lq.gemm_i8_plan(4, 64, 64, 2 ** 32 + 1)]
    for call in calls:
        with pytest.raises(ValueError, match="exceeds 32 bits"):
            call()
    assert not rec.calls


@pytest.mark.parametrize("gate_tokens", [8, 100, 2 ** 31, 2 ** 32 + 1, 2 ** 40])
def test_one_gate_row_for_any_number_of_tokens(rec, gate_tokens):
    """Cut down to 32 bits, 2^32 + 1 would send token t to row t of a gate of one row."""
    h, gate = torch.zeros(8, 64), torch.zeros(1, 64)
    lq.norm_residual(h, gate=gate, gate_tokens=gate_tokens)
    d = descriptor(rec.calls[-1], lq.GateDesc)
    assert d.cols == 64 and d.gate == gate.data_ptr()
    assert all(t // d.tokens == 0 for t in range(8))


def test_gate_rows(rec):
    h = torch.zeros(8, 64)
    for shape, given, tokens in (((64,), 0, 8), ((1, 64), 0, 8), ((8, 64), 0, 1), ((8, 1), 0, 1),
                                 ((3, 64), 3, 3), ((2, 1), 7, 7)):
        lq.norm_residual(h, gate=torch.zeros(shape), gate_tokens=given)
        d = descriptor(rec.calls[-1], lq.GateDesc)
        assert (d.tokens, d.cols) == (tokens, shape[-1])
    for shape, given in (((2, 64), 0), ((9, 64), 1), ((3, 64), 4), ((1, 64), -1)):
        with pytest.raises(ValueError, match="does not give"):
            lq.norm_residual(h, gate=torch.zeros(shape), gate_tokens=given)
    assert ctypes.sizeof(lq.GateDesc) == 24


@pytest.mark.parametrize("shape,given", [((0, 64), 0), ((0, 64), 1), ((0, 1), 3), ((1, 64), 0),
                                         ((64,), 0), ((1, 1), 8)])
def test_gate_of_an_empty_batch(rec, shape, given):
    """A gate row per token is an empty gate where there are no tokens."""
    c, n = lq.norm_residual(torch.zeros(0, 64), torch.zeros(0, 64), gate=torch.zeros(shape),
                            gate_tokens=given)
    assert c.shape == n.shape == (0, 64) and descriptor(rec.calls[-1], lq.GateDesc).tokens >= 1
    with pytest.raises(ValueError, match="does not give"):
        lq.norm_residual(torch.zeros(0, 64), gate=torch.zeros(2, 64), gate_tokens=given)


def test_residual_out_over_inputs(rec):
    """In place or apart; what would overwrite rows before they are read is refused."""
    rows, K = 6, 64
    buf = torch.zeros(4 * rows * K)
    view = lambda at, step=K, n=rows: buf.as_strided((n, K), (step, 1), at)  # noqa: E731
    h, r = torch.zeros(rows, K), view(0)
    strided = view(0, 2 * K)
    for h_, r_, out in ((h, r, r), (h, r, view(0)), (h, strided, strided), (h, r, view(rows * K)),
                        (h, strided, view(2 * rows * K)), (r, None, view(0)), (r, view(rows * K), r),
                        (strided, view(K, 2 * K), None), (h, None, view(5))):
        lq.norm_residual(h_, r_, residual_out=out)
    inside = view(K, 2 * K)         # every other row of the same memory
    lq.norm_residual(strided, inside, residual_out=inside)
    calls = len(rec.calls)
    for h_, r_, out, name in ((h, r, view(K), "residual"), (h, view(K), view(0), "residual"),
                              (h, strided, view(0), "residual"), (h, strided, view(K), "residual"),
                              (view(8), None, view(0), "h"), (strided, None, view(0), "h"),
                              (h, r, view(1), "residual"),
                              (r, view(2 * rows * K), view(K), "h")):
        with pytest.raises(ValueError, match="residual_out overlaps " + name):
            lq.norm_residual(h_, r_, residual_out=out)
    with pytest.raises(ValueError, match="residual_out overlaps h"):
        lq.norm_residual(view(8, 2 * K), strided, residual_out=strided)
    half = buf.view(torch.bfloat16)[:rows * K].view(rows, K)
    with pytest.raises(ValueError, match="residual_out overlaps h"):
        lq.norm_residual(half, None, residual_out=r)
    assert len(rec.calls) == calls
    empty = torch.zeros(0, K)
    lq.norm_residual(empty, empty, residual_out=torch.zeros(0, K))


def test_import_with_a_cpu_build_of_torch():
    """The host-only queries need no CUDA in torch."""
    code = ("import torch\n"
            "for name in [n for n in vars(torch._C) if n.startswith('_cuda')]:\n"
            "    delattr(torch._C, name)\n"
            "import fractional_bit_weight_b200 as lq\n"
            "assert lq.gemm_route(1, 4096, 4096, 10, 24) >= 0\n"
            "assert lq.gemm_i8_route(1, 4096, 4096) >= 0\n"
            "try:\n"
            "    lq.quant_i8(torch.zeros(2, 64))\n"
            "except TypeError:\n"
            "    print('refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(lq.__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "refused", out.stderr


def test_parts_of_t_without_t(rec):
    """sign and chan_scale belong to T: with block = 0 they would be dropped without a word."""
    x, sign, scale = torch.zeros(4, 64), torch.ones(64, dtype=torch.int8), torch.ones(64)
    for parts in (dict(sign=sign), dict(chan_scale=scale), dict(sign=sign, chan_scale=scale)):
        for call in (lambda **kw: lq.quant_i8(x, **kw), lambda **kw: lq.norm_residual_i8(x, **kw)):
            with pytest.raises(ValueError, match="block = 0"):
                call(**parts)
            assert not rec.calls
            call(**parts, block=1)
            d = descriptor(rec.calls.pop(), lq.WhitenDesc)
            assert d.block == 1
            assert d.sign == (sign.data_ptr() if "sign" in parts else None)
            assert d.chan_scale == (scale.data_ptr() if "chan_scale" in parts else None)
    lq.quant_i8(x)
    lq.norm_residual_i8(x)


def test_calls_without_a_workspace_share_one(rec, monkeypatch):
    """The status word of a call that is given no workspace is where default_i8_workspace() says."""
    capturing = [True]
    stream = type("Stream", (), {"synchronize": lambda self: None})()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(lq, "_I8_WORKSPACES", {}, raising=False)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.ones(4)

    def workspace_of(**kw):
        lq.gemm_i8(q, s, q, s, **kw)
        return rec.calls[-1][1][10]

    workspace_of()
    assert not lq._I8_WORKSPACES    # a captured call's workspace belongs to its graph
    capturing[0] = False
    at = workspace_of()
    assert at == workspace_of() == lq._I8_WORKSPACES[HOST].data_ptr()
    capturing[0] = True
    assert at == workspace_of()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: HOST)
    assert at == lq.default_i8_workspace().data_ptr()
    own = torch.zeros(256, dtype=torch.uint8)
    assert workspace_of(workspace=own) == own.data_ptr()
