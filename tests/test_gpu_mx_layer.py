"""The MXFP4 layer as it is used: norm, product and their gradients together,
eager, in captured graphs and on several streams; the example; what the binding
refuses."""

import importlib.util
import os
import warnings

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer, mx
from tests.gpu_util import assert_bits_equal, bits, case, dev, torch
from tests.test_gpu_int8 import DT, make, tdt, upload
from tests.test_gpu_mxfp4 import within

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Step:
    """Forward and backward of norm and linear layer with workspaces and outputs of its own."""

    def __init__(self, t, M, N, K, seed=0, device=None, workspace=None):
        T = torch()
        self.t, self.M, self.N, self.K = t, M, N, K
        self.dev = device or dev()
        rng = np.random.default_rng(seed)
        make_one = lambda shape, spread: upload(make(rng, shape, t, spread)[0], t)  # noqa: E731
        self.x, self.g, self.w = make_one((M, K), 1.0), make_one((M, N), 1.0), make_one((N, K), 0.3)
        self.nw = T.from_numpy((1 + 0.1 * rng.standard_normal(K)).astype(np.float32)).to(self.dev)
        self.nb = T.from_numpy((0.1 * rng.standard_normal(K)).astype(np.float32)).to(self.dev)
        self.bias = upload(layer.round_to(rng.standard_normal((1, N)).astype(np.float32), t), t)[0]
        lib = kb.lib()
        need = max(lib.linear_mxfp4_dynamic_workspace_bytes(M, N, K), lib.linear_mxfp4_backward_workspace_bytes(M, N, K),
                   lib.layer_norm_backward_workspace_bytes(M, K))
        self.ws = T.full((need,), 0xFF, dtype=T.uint8, device=self.dev) if workspace is None else workspace
        self.codes = T.empty((N, -(-K // 32) * 16), dtype=T.uint8, device=self.dev)
        self.scales = T.empty((N, -(-K // 32)), dtype=T.uint8, device=self.dev)
        self.y, self.dy, self.dx = (T.empty_like(self.x) for _ in range(3))
        self.out = T.empty((M, N), dtype=tdt(t), device=self.dev)
        self.dw = T.empty((N, K), dtype=T.float32, device=self.dev)

    def run(self):
        kb.layer_norm(self.x, self.nw, self.nb, out=self.y)
        kb.quantize_mxfp4(self.w, self.codes, self.scales)
        kb.linear_mxfp4_dynamic(self.y, self.codes, self.scales, bias=self.bias, out=self.out, workspace=self.ws)
        _, _, self.db = kb.linear_mxfp4_backward(self.g, self.y, self.w, dX=self.dy, dweight=self.dw, workspace=self.ws)
        _, self.dnw, self.dnb = kb.layer_norm_backward(self.dy, self.x, self.nw, dx=self.dx, workspace=self.ws)

    NAMES = ("y", "codes", "scales", "out", "dy", "dw", "db", "dx", "dnw", "dnb")

    def outputs(self):
        return {n: bits(getattr(self, n)) for n in self.NAMES}

    def clear(self):
        for n in self.NAMES:
            getattr(self, n).fill_(3)


def same(got, want, what):
    for n in Step.NAMES:
        assert_bits_equal(got[n], want[n], f"{what}: {n}")


SIZES = [("bf16", 1, 96, 128), ("bf16", 5, 300, 520), ("fp32", 65, 130, 777), ("fp16", 300, 512, 640), ("bf16", 2100, 1030, 2056),
         ("bf16", 2304, 4096, 2048)]


@pytest.mark.parametrize("t,M,N,K", SIZES)
def test_together(t, M, N, K):
    # each stage against the formula on what the one before it gave
    case(f"mx layer {t} M={M} N={N} K={K}")
    s = Step(t, M, N, K)
    s.run()

    def val(v):
        return v.float().cpu().numpy()
    x, y, g, w, nw, nb = (val(v) for v in (s.x, s.y, s.g, s.w, s.nw, s.nb))
    within(s.y, *mx.layer_norm(x, nw, nb, 1e-5), t, "norm")
    for got, want in zip((s.codes, s.scales), mx.quantize(w)):
        assert_bits_equal(got.cpu().numpy(), want, "weight")
    within(s.out, *mx.product(mx.rounded(y), mx.rounded(w), val(s.bias)), t, "product")
    (dy, ey), (dw, ew), (db, eb) = mx.linear_backward(g, y, w)
    within(s.dy, dy, ey, t, "dy")
    within(s.dw, dw, ew, "fp32", "dw")
    within(s.db, db, eb, "fp32", "db")
    for got, (v, e), ty in zip((s.dx, s.dnw, s.dnb), mx.layer_norm_back(val(s.dy), x, nw, 1e-5), (t, "fp32", "fp32")):
        within(got, v, e, ty, "norm's gradient")


@pytest.mark.parametrize("t,M,N,K", SIZES)
def test_replayed(t, M, N, K):
    # two graphs that share a workspace, replayed in turn with new inputs, with
    # eager work in the same workspace in between
    T = torch()
    case(f"mx layer captured {t} M={M} N={N} K={K}")
    a = Step(t, M, N, K)
    b = Step(t, M, N, K, seed=1, workspace=a.ws)
    eager = Step(t, M, N, K, seed=2, workspace=a.ws)
    for s in (a, b, eager):
        s.run()
    T.cuda.synchronize()
    graphs = []
    for s in (a, b):
        g = T.cuda.CUDAGraph()
        with T.cuda.graph(g):
            s.run()
        graphs.append(g)
    for r in range(3):
        for s, g in zip((a, b), graphs):
            case(f"replay {r}")
            s.x.mul_(-0.5)
            s.g.mul_(2)
            s.w.add_(0.25)
            s.clear()
            a.ws.fill_(0xFF)
            g.replay()
            T.cuda.synchronize()
            got = s.outputs()
            eager.x.copy_(s.x), eager.g.copy_(s.g), eager.w.copy_(s.w)
            eager.nw.copy_(s.nw), eager.nb.copy_(s.nb), eager.bias.copy_(s.bias)
            eager.run()
            T.cuda.synchronize()
            same(got, eager.outputs(), f"replay {r}")


def test_replayed_without_given_memory():
    # workspaces and outputs from the capture's own pool
    T = torch()
    M, N, K = 2304, 1100, 2056
    x, g, w = (T.randn(s, device=dev(), dtype=T.bfloat16) for s in ((M, K), (M, N), (N, K)))
    nw = T.ones(K, device=dev())

    def step():
        y = kb.layer_norm(x, nw)
        out = kb.linear_mxfp4_dynamic(y, *kb.quantize_mxfp4(w))
        dy, dw, db = kb.linear_mxfp4_backward(g, y, w)
        return (out, dw, db, *kb.layer_norm_backward(dy, x, nw, dx=dy))
    case("mx layer captured without given memory")
    step()
    T.cuda.synchronize()
    graph = T.cuda.CUDAGraph()
    with T.cuda.graph(graph):
        held = step()
    for r in range(3):
        x.neg_()
        g.mul_(0.5)
        graph.replay()
        T.cuda.synchronize()
        got = [bits(v) for v in held]
        for a, b in zip(got, step()):
            assert_bits_equal(a, bits(b), f"replay {r}")


@pytest.mark.parametrize("t,M,N,K", [("bf16", 5, 300, 520), ("fp16", 300, 512, 640), ("bf16", 2304, 4096, 2048)])
def test_two_at_once(t, M, N, K):
    # on two streams that are not the current one, each behind its own inputs
    T = torch()
    case(f"mx layer on two streams {t} M={M} N={N} K={K}")
    steps = [Step(t, M, N, K, seed=i) for i in range(2)]
    want = []
    for s in steps:
        s.run()
        want.append(s.outputs())
        s.clear()
    streams = [T.cuda.Stream() for _ in steps]
    T.cuda.synchronize()
    for r in range(3):
        for s, stream in zip(steps, streams):
            with T.cuda.stream(stream):
                s.ws.fill_(0xFF)
                s.run()
    for stream in streams:
        stream.synchronize()
    for s, w in zip(steps, want):
        same(s.outputs(), w, "two streams")


def test_the_same_tensor_twice():
    # operands that are one tensor, or views of one
    T = torch()
    x = T.randn(320, 320, device=dev(), dtype=T.bfloat16)
    codes, scales = kb.quantize_mxfp4(x)
    case("mx operands twice")
    got = kb.linear_mxfp4(codes, scales, codes, scales, dtype=T.float32)
    v = mx.rounded(x.float().cpu().numpy())
    within(got, *mx.product(v, v), "fp32", "codes twice")
    got = kb.linear_mxfp4(codes[10:20], scales[10:20], codes[15:], scales[15:], dtype=T.float32)
    within(got, *mx.product(v[10:20], v[15:]), "fp32", "views of one")
    for got, (want, e), ty in zip(kb.linear_mxfp4_backward(x, x, x), mx.linear_backward(*(x.float().cpu().numpy(),) * 3),
                                  ("bf16", "fp32", "fp32")):
        within(got, want, e, ty, "one tensor three times")
    w = T.ones(320, device=dev(), dtype=T.bfloat16)
    for got, (want, e), ty in zip(kb.layer_norm_backward(x, x, w), mx.layer_norm_back(
            *(x.float().cpu().numpy(),) * 2, np.ones(320), 1e-5), ("bf16", "fp32", "fp32")):
        within(got, want, e, ty, "dout is x")


def example():
    spec = importlib.util.spec_from_file_location("mx_layer", os.path.join(ROOT, "examples", "mx_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("args", [["--tokens", "300", "--hidden", "512", "--layers", "2", "--steps", "2"],
                                  ["--tokens", "33", "--hidden", "200", "--layers", "1", "--steps", "1"]])
def test_example(args):
    case(f"mx layer example {args}")
    net, x, alone, whole = example().main(args)
    assert alone.shape == whole.shape and torch().isfinite(alone.float()).all()
    assert all(p.grad is not None and torch().isfinite(p.grad.float()).all() for p in net.parameters())
    if len(net) == 1:  # the same codes: sums of 200 products in two orders, then bf16 twice
        one = net[0]
        y = kb.layer_norm(x[:4], one.norm_weight.detach(), one.norm_bias.detach()).float().cpu().numpy()
        w = mx.values(one.codes.cpu().numpy(), one.scales.cpu().numpy(), 200)
        p, e = mx.product(mx.rounded(y), w, one.bias.detach().float().cpu().numpy())
        e = e + 2.0 ** -8 * (np.abs(p) + e)
        limit = e + 2.0 ** -8 * (np.abs(p + x[:4].float().cpu().numpy()) + e)
        for v in (alone, whole):
            assert (np.abs(v.double().cpu().numpy() - p - x[:4].double().cpu().numpy()) <= limit).all()


@pytest.mark.parametrize("M,K", [(40, 64), (130, 257)])
def test_gradients_of_the_example(M, K):
    T = torch()
    case(f"mx layer example's gradients {M}x{K}")
    T.manual_seed(1)
    one = example().MxLayer(K)
    x = T.randn(M, K, device=dev(), dtype=T.bfloat16, requires_grad=True)
    g = T.randn(M, K, device=dev(), dtype=T.bfloat16)
    with warnings.catch_warnings():
        warnings.simplefilter("error")  # nothing is cut off
        one(x).backward(g)

    def val(v):
        return v.detach().float().cpu().numpy()
    y = val(kb.layer_norm(x.detach(), one.norm_weight.detach(), one.norm_bias.detach()))
    (dy, ey), (dw, ew), (db, eb) = mx.linear_backward(val(g), y, val(one.weight))
    within(one.weight.grad, dw, ew + 2.0 ** -24 * np.abs(dw), "bf16", "weight")
    within(one.bias.grad, db, eb + 2.0 ** -24 * np.abs(db), "bf16", "bias")
    # dy as the kernels give it, checked by its own bound above the norm's
    got = kb.linear_mxfp4_backward(g, T.from_numpy(y).to(dev()).bfloat16(), one.weight.detach())[0]
    within(got, dy, ey, "bf16", "dy")
    (dx, ex), (dnw, enw), (dnb, enb) = mx.layer_norm_back(val(got), val(x), val(one.norm_weight), 1e-5)
    within(one.norm_weight.grad, dnw, enw, "fp32", "norm_weight")
    within(one.norm_bias.grad, dnb, enb, "fp32", "norm_bias")
    # through the norm in bf16, then added to the residual's gradient in bf16
    e = ex + 2.0 ** -8 * (np.abs(dx) + ex)
    within(x.grad, dx + val(g), e, "bf16", "x")


def bad(exc, match, fn, *a, **kw):
    with pytest.raises(exc, match=match):
        fn(*a, **kw)


def test_refusals():
    T = torch()
    u8 = dict(dtype=T.uint8, device=dev())
    x = T.randn(8, 64, device=dev(), dtype=T.bfloat16)
    c, s = kb.quantize_mxfp4(x)
    w = T.ones(64, device=dev(), dtype=T.bfloat16)
    case("mx refusals")
    # quantize, dequantize
    bad(ValueError, "contiguous", kb.quantize_mxfp4, T.as_strided(x, (2, 3), (100, 2)))
    bad(ValueError, "overlap", kb.quantize_mxfp4, T.as_strided(x, (8, 64), (60, 1)))
    bad(ValueError, "overlap", kb.quantize_mxfp4, T.as_strided(x, (64, 7), (1, 60)))
    bad(ValueError, "between 1 and", kb.quantize_mxfp4, x[:, :0])
    bad(ValueError, "rows of 16 bytes", kb.quantize_mxfp4, x, c[:, :16], s)
    bad(ValueError, "scales", kb.quantize_mxfp4, x, c, s[:4])
    bad(ValueError, "rows", kb.quantize_mxfp4, x[:7], c, s)
    bad(TypeError, "codes", kb.quantize_mxfp4, x, x, s)
    bad(ValueError, "overlaps X", kb.quantize_mxfp4, x, x.view(T.uint8)[:, :32], s)
    pool = T.empty(8 * 48, **u8)
    bad(ValueError, "codes overlaps scales", kb.quantize_mxfp4, x, pool.view(8, 48)[:, :32], pool.view(8, 48)[:, 31:33])
    kb.quantize_mxfp4(x, pool.view(8, 48)[:, :32], pool.view(8, 48)[:, 32:34])  # beside each other is fine
    bad((ValueError, kb.KbitError), "quantize_mxfp4", kb.quantize_mxfp4, x, T.empty(8 * 40, **u8).view(8, 40)[:, :32], s)  # rows 40 bytes apart
    bad(ValueError, "rows of 32 bytes", kb.dequantize_mxfp4, c, s, 65)
    bad(ValueError, "out", kb.dequantize_mxfp4, c, s, 64, out=T.empty(8, 63, device=dev(), dtype=T.bfloat16))
    bad(TypeError, "out", kb.dequantize_mxfp4, c, s, 64, out=T.empty(8, 64, device=dev()))
    # products
    for fn in (lambda **k: kb.linear_mxfp4(c, s, k.pop("wc", c), k.pop("ws", s), **k),
               lambda **k: kb.linear_mxfp4_dynamic(x, k.pop("wc", c), k.pop("ws", s), **k)):
        bad(ValueError, "w_codes", fn, wc=T.empty(8, 48, **u8))
        bad(ValueError, "w_scales", fn, ws=T.empty(8, 3, **u8))
        bad(TypeError, "w_scales", fn, ws=T.empty(8, 2, device=dev()))
        bad(ValueError, "at least one row", fn, wc=c[:0], ws=s[:0])
        bad(ValueError, "bias: 64 elements", fn, bias=w)
        bad(TypeError, "bias", fn, bias=T.zeros(8, device=dev()))
        bad(ValueError, "out", fn, out=T.empty(8, 9, device=dev(), dtype=T.bfloat16))
        bad(TypeError, "out", fn, out=T.empty(8, 8, device=dev()))
        bad(ValueError, "overlap", fn, out=T.empty(100, device=dev(), dtype=T.bfloat16).as_strided((8, 8), (7, 1)))
        bad(ValueError, "out overlaps w_scales", fn, ws=pool[:16].view(8, 2), out=pool[8:8 + 128].view(T.bfloat16).view(8, 8))
        bad(ValueError, "live on|same device|device", fn, wc=c.cpu())
    bad(ValueError, "out overlaps X", lambda: kb.linear_mxfp4_dynamic(x, c, s, out=x[:, :8]))
    bad(ValueError, "out overlaps codes", lambda: kb.linear_mxfp4(c, s, *kb.quantize_mxfp4(x.clone()), out=c.view(T.bfloat16)[:, :8]))
    bad(ValueError, "whole blocks", kb.linear_mxfp4, c[:, :24], s, c, s)
    need = kb.lib().linear_mxfp4_dynamic_workspace_bytes(300, 8, 64)
    many = T.randn(300, 64, device=dev(), dtype=T.bfloat16)
    bad(ValueError, "workspace", kb.linear_mxfp4_dynamic, many, c, s, workspace=T.empty(need - 1, **u8))
    bad(TypeError, "workspace", kb.linear_mxfp4_dynamic, many, c, s, workspace=T.empty(need, device=dev()))
    kb.linear_mxfp4_dynamic(many, c, s, workspace=T.empty(need, **u8))
    # gradients
    g = T.randn(8, 16, device=dev(), dtype=T.bfloat16)
    wt = T.randn(16, 64, device=dev(), dtype=T.bfloat16)
    back = kb.linear_mxfp4_backward
    bad(ValueError, "X", back, g, x[:7], wt)
    bad(ValueError, "weight", back, g, x, wt[:, :63])
    bad(TypeError, "X", back, g, x.float(), wt)
    bad(TypeError, "weight", back, g, x, wt.half())
    bad(ValueError, "not asked for", back, g, x, wt, input_grad=False, dX=T.empty_like(x))
    bad(ValueError, "not asked for", back, g, x, wt, weight_grad=False, dweight=T.empty(16, 64, device=dev()))
    bad(ValueError, "dX overlaps X", back, g, x, wt, dX=x)
    bad(TypeError, "dweight", back, g, x, wt, dweight=T.empty_like(wt))
    both = T.empty(8 * 64 * 2 + 16 * 64 * 4, **u8)
    bad(ValueError, "dweight overlaps dX", back, g, x, wt, dX=both[:1024].view(T.bfloat16).view(8, 64),
        dweight=both[512:512 + 4096].view(T.float32).view(16, 64))
    bad(ValueError, "workspace", back, g, x, wt, workspace=T.empty(100, **u8))
    # norm
    bad(ValueError, "63 elements, at least 64", kb.layer_norm, x, w[:63])
    bad(ValueError, "must have 64 elements", kb.layer_norm, x, T.ones(65, device=dev()))
    bad(TypeError, "weight", kb.layer_norm, x, w.half())
    bad(TypeError, "bias", kb.layer_norm, x, w, w.float())
    bad(ValueError, "one column", kb.layer_norm, x[:, :0], w[:0])
    bad((ValueError, kb.KbitError), "layer_norm", kb.layer_norm, x, w, eps=-1.0)
    bad(ValueError, "out", kb.layer_norm, x, w, out=x[:, :63])
    bad(ValueError, "overlap", kb.layer_norm, x[:7], w, out=x[1:])
    bad(ValueError, "out overlaps weight", kb.layer_norm, x[:1], w, out=w[None])
    nb = kb.layer_norm_backward
    bad(ValueError, "dout", nb, x[:7], x, w)
    bad(TypeError, "dout", nb, x.float(), x, w)
    bad(ValueError, "dx overlaps x", nb, x.clone(), x, w, dx=x)
    bad(ValueError, "overlap", nb, x[:7], x[:7].clone(), w, dx=x[1:])
    bad(ValueError, "workspace", nb, x, x.clone(), w, workspace=T.empty(64, **u8))


def test_written_tensors_count_as_modified():
    T = torch()
    x = T.randn(8, 64, device=dev())
    c, s = kb.quantize_mxfp4(x)
    out, dx, y, dn = T.empty(8, 8, device=dev()), *(T.empty_like(x) for _ in range(3))
    dw = T.empty(8, 64, device=dev())
    case("mx outputs count as modified")
    before = {n: v._version for n, v in dict(c=c, s=s, out=out, dx=dx, dw=dw, y=y, dn=dn, x=x).items()}
    kb.quantize_mxfp4(x, c, s)
    kb.linear_mxfp4(c, s, c, s, dtype=T.float32, out=out)
    kb.linear_mxfp4_backward(out, x, x, dX=dx, dweight=dw)
    kb.layer_norm(x, x[0], out=y)
    kb.layer_norm_backward(x, x, x[0], dx=dn)
    after = dict(c=c, s=s, out=out, dx=dx, dw=dw, y=y, dn=dn, x=x)
    for n, v in after.items():
        assert (v._version > before[n]) == (n != "x"), n


def test_a_gradient_that_is_cut_off_is_said():
    T = torch()
    x = T.randn(8, 64, device=dev(), requires_grad=True)
    d = x.detach()
    c, s = kb.quantize_mxfp4(d)
    w = T.ones(64, device=dev())
    for call in (lambda: kb.quantize_mxfp4(x), lambda: kb.linear_mxfp4_dynamic(x, c, s), lambda: kb.layer_norm(x, w),
                 lambda: kb.linear_mxfp4_backward(x, d, T.ones(64, 64, device=dev())),
                 lambda: kb.layer_norm_backward(d, x, w), lambda: kb.linear_mxfp4(c, s, c, s, bias=x[0, :8].contiguous(), dtype=T.float32)):
        with pytest.warns(UserWarning, match="requires a gradient"):
            call()
        with warnings.catch_warnings(), T.no_grad():
            warnings.simplefilter("error")
            call()
