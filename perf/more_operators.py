"""Cases of microscaled 4-bit linear layers (MXFP4) and of the layer norm in
front of them, for training and serving, in their plain form and through the
framework's entry points.

MXFP4: blocks of 32 values with one power of two each, 2^(floor(log2(max)) - 2)
held as a byte, and codes of 4 bits, a sign and a magnitude of 0, 1/2, 1, 3/2, 2,
3, 4 or 6 (nearest, ties to the even code, at most 6).

* ``quantize``  rows of a matrix, or of its transpose, to codes and scales, and
  the values they stand for;
* ``linear``    out = x W^T + bias with both operands in MXFP4; x is quantized
  on the way ("values") or comes as codes already ("codes");
* ``back``      a training step's gradients of such a layer: input, weight and
  bias, from the products of dout, x and W quantized along the axes that those
  sum over;
* ``norm``      layer norm of rows;
* ``normback``  its gradients: input, weight and bias.

``own = False`` computes with elementary torch operations in fp32, rounded
once at the end; ``own = True`` calls the framework.
"""

import math

import torch

own = False

_DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
_EPS = 1e-5

# The largest listed passes: no drawn case costs more.
_MAX_MNK = 8192 * 11008 * 4096
_MAX_BACK_MNK = 8192 * 4096 * 4096
_MAX_ELEMS = 8192 * 11008
_MAX_NORM_ELEMS = 8192 * 4096


def listed():
    return [
        # a whole prompt's activations into codes, row by row
        dict(name="quantize-prompt", op="quantize", dtype="bf16", rows=8192, d=11008, columns=False),
        # an odd fp32 matrix along its columns, as a weight's gradient needs its operands
        dict(name="quantize-columns", op="quantize", dtype="fp32", rows=2731, d=4099, columns=True),
        # one token through a square projection: the weight read and the launch
        dict(name="linear-token", op="linear", dtype="bf16", input="values", M=1, N=4096, K=4096, bias=False),
        # an uneven decode batch through a wide layer, fp16 with a bias
        dict(name="linear-batch", op="linear", dtype="fp16", input="values", M=77, N=11008, K=4096, bias=True),
        # a chunk of a prompt whose codes are shared by several projections;
        # odd channels, and a depth that is no whole number of steps
        dict(name="linear-chunk", op="linear", dtype="fp32", input="codes", M=500, N=4099, K=3800, bias=False),
        # a whole prompt through the wide layer
        dict(name="linear-prompt", op="linear", dtype="bf16", input="values", M=8192, N=11008, K=4096, bias=False),
        # gradients of a small uneven layer in fp16
        dict(name="back-small", op="back", dtype="fp16", M=333, N=1000, K=1031),
        # gradients of a square projection over a batch of sequences
        dict(name="back-train", op="back", dtype="bf16", M=8192, N=4096, K=4096),
        # a decode batch
        dict(name="norm-batch", op="norm", dtype="bf16", rows=16, d=4096, weight="same"),
        # a prompt, an odd number of rows
        dict(name="norm-prompt", op="norm", dtype="bf16", rows=8191, d=4096, weight="same"),
        # a small fp32 layer of odd width
        dict(name="normback-odd", op="normback", dtype="fp32", rows=700, d=1025, weight="same"),
        # a training step's gradients, 16-bit values with fp32 weights
        dict(name="normback-train", op="normback", dtype="bf16", rows=8192, d=4096, weight="fp32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "back", "norm", "normback"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    half = 2 if dtype == "fp32" else 1
    if op == "quantize":
        d = _log(rng, 32, 16384)
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(8192, _MAX_ELEMS // half // d)), d=d,
                    columns=rng.random() < 0.5)
    if op in ("linear", "back"):
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 64, 16384), _log(rng, 64, 16384)
            if rng.random() < 0.6:  # most layers have even widths, some do not
                N, K = -(-N // 64) * 64, -(-K // 64) * 64
            if M * N * K > (_MAX_MNK if op == "linear" else _MAX_BACK_MNK):
                continue
            if op == "back":
                if max(M * N, M * K, N * K) <= _MAX_NORM_ELEMS // half:
                    return dict(op=op, dtype=dtype, M=M, N=N, K=K)
                continue
            return dict(op=op, dtype=dtype, input=rng.choice(["values", "codes"]), M=M, N=N, K=K,
                        bias=rng.random() < 0.5)
    d = _log(rng, 64, 16384)
    if rng.random() < 0.6:
        d = -(-d // 64) * 64
    return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(16384, _MAX_NORM_ELEMS // half // d)), d=d,
                weight=rng.choice(["same", "fp32"]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _activations(g, rows, d):
    """Tokens of different magnitude, a few channels of which stand out."""
    x = torch.randn((rows, d), generator=g, device="cuda")
    x *= torch.exp(torch.rand((rows, 1), generator=g, device="cuda") * 4.0 - 2.0)
    out = torch.rand(d, generator=g, device="cuda") < 0.01
    return torch.where(out, x * 12.0, x)


def _weight(g, rows, d):
    return torch.randn((rows, d), generator=g, device="cuda") * 0.02


def _inputs(case, seed):
    """The data of a case, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op = _DT[case["dtype"]], case["op"]
    if op == "quantize":
        return {"x": _activations(g, case["rows"], case["d"]).to(dt)}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(g, M, K).to(dt)
        d = {"x": x} if case["input"] == "values" else dict(zip(("codes", "scales"), _codes(x)))
        d["w_codes"], d["w_scales"] = _codes(_weight(g, N, K))
        d["bias"] = torch.randn(N, generator=g, device="cuda").to(dt) if case["bias"] else None
        return d
    if op == "back":
        M, N, K = case["M"], case["N"], case["K"]
        return {"x": _activations(g, M, K).to(dt), "weight": _weight(g, N, K).to(dt),
                "dout": (torch.randn((M, N), generator=g, device="cuda") * 0.05).to(dt)}
    R, D = case["rows"], case["d"]
    # rows whose mean is not zero
    x = _activations(g, R, D) + torch.randn((R, 1), generator=g, device="cuda")
    wt = torch.float32 if case["weight"] == "fp32" else dt
    d = {"x": x.to(dt), "weight": (1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(wt),
         "bias": (0.1 * torch.randn(D, generator=g, device="cuda")).to(wt)}
    if op == "normback":
        d["dout"] = torch.randn((R, D), generator=g, device="cuda").to(dt)
    return d


def prepare(case, seed):
    return dict(case=case, **_inputs(case, seed))


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _blocks(x):
    """x fp32 [rows, d] as [rows, blocks, 32], zeros past d."""
    rows, d = x.shape
    return torch.nn.functional.pad(x, (0, -d % 32)).view(rows, -1, 32)


def _plain_quantize(x):
    """(scaled values [rows, blocks, 32] rounded to what a code can be, scale
    bytes [rows, blocks])."""
    b = _blocks(x.float())
    _, e = torch.frexp(b.abs().amax(-1))  # max = m 2^e, 1/2 <= m < 1
    e = torch.where(b.abs().amax(-1) == 0, -127, e - 3).clamp(min=-127)
    y = torch.ldexp(b, -e[..., None])
    a = y.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.where(y < 0, -q, q), (e + 127).to(torch.uint8)


def _codes(x):
    """Two codes a byte, the first in the low half, whole blocks a row; and the
    scale bytes."""
    q, s = _plain_quantize(x)
    a = q.abs()
    c = torch.where(a < 2.0, 2.0 * a, torch.where(a < 4.0, a + 2.0, a / 2.0 + 4.0)).to(torch.uint8)
    c += 8 * (q < 0).to(torch.uint8)
    c = c.view(x.shape[0], -1, 2)
    return (c[..., 0] + 16 * c[..., 1]).contiguous(), s


def _decode(codes, scales):
    """fp32 [rows, 32 blocks]"""
    c = torch.stack([codes & 15, codes >> 4], -1).view(*scales.shape, 32)
    m = (c & 7).float()
    v = torch.where(m < 4.0, m * 0.5, torch.where(m < 6.0, m - 2.0, 2.0 * m - 8.0))
    v = torch.where(c > 7, -v, v)
    return torch.ldexp(v, scales.to(torch.int32)[..., None] - 127).flatten(1)


def _values(x, d=None):
    """What the codes of x's rows stand for, fp32."""
    q, s = _plain_quantize(x)
    v = torch.ldexp(q, s.to(torch.int32)[..., None] - 127).flatten(1)
    return v if d is None else v[:, :d]


def _plain(s):
    c = s["case"]
    op, dt = c["op"], _DT[c["dtype"]]
    if op == "quantize":
        x = s["x"].t() if c["columns"] else s["x"]
        q, sc = _plain_quantize(x)
        v = torch.ldexp(q, sc.to(torch.int32)[..., None] - 127).flatten(1)[:, :x.shape[1]]
        return [v.to(dt), sc]
    if op == "linear":
        x = _values(s["x"]) if c["input"] == "values" else _decode(s["codes"], s["scales"])
        y = x @ _decode(s["w_codes"], s["w_scales"]).t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y.to(dt)
    if op == "back":
        dx = _values(s["dout"]) @ _values(s["weight"].t()).t()
        dw = _values(s["dout"].t()) @ _values(s["x"].t()).t()
        return [dx.to(dt), dw, s["dout"].float().sum(0)]
    x, w = s["x"].float(), s["weight"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    r = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + _EPS)
    xhat = xc * r
    if op == "norm":
        return (xhat * w + s["bias"].float()).to(dt)
    g = s["dout"].float()
    h = g * w
    dx = r * (h - h.mean(-1, keepdim=True) - xhat * (h * xhat).mean(-1, keepdim=True))
    return [dx.to(dt), (g * xhat).sum(0), g.sum(0)]


def _own(s):
    import blockwise_bit_codebook_amd as kb
    c = s["case"]
    op, dt = c["op"], _DT[c["dtype"]]
    if op == "quantize":
        x = s["x"].t() if c["columns"] else s["x"]
        codes, scales = kb.quantize_mxfp4(x)
        return [kb.dequantize_mxfp4(codes, scales, x.shape[1], dtype=dt), scales]
    if op == "linear":
        if c["input"] == "codes":
            return kb.linear_mxfp4(s["codes"], s["scales"], s["w_codes"], s["w_scales"], bias=s["bias"], dtype=dt)
        return kb.linear_mxfp4_dynamic(s["x"], s["w_codes"], s["w_scales"], bias=s["bias"])
    if op == "back":
        return list(kb.linear_mxfp4_backward(s["dout"], s["x"], s["weight"]))
    if op == "norm":
        return kb.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS)
    return list(kb.layer_norm_backward(s["dout"], s["x"], s["weight"], eps=_EPS))


def run(state):
    return _own(state) if own else _plain(state)


def _packed(rows, d):
    """Bytes of rows in MXFP4."""
    return rows * -(-d // 32) * 17


def work(case):
    """Inputs once, outputs once."""
    e, op = _SIZE[case["dtype"]], case["op"]
    if op == "quantize":
        n = case["rows"] * case["d"]
        packed = _packed(case["d"], case["rows"]) if case["columns"] else _packed(case["rows"], case["d"])
        return {"bytes": 2 * n * e + packed, "flops": 4 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = _packed(M, K) if case["input"] == "codes" else M * K * e
        return {"bytes": x + _packed(N, K) + (N * e if case["bias"] else 0) + M * N * e, "flops": 2 * M * N * K}
    if op == "back":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M * N + 2 * M * K + N * K) * e + 4 * (N * K + N), "flops": 4 * M * N * K}
    n, d = case["rows"] * case["d"], case["d"]
    w = 4 if case["weight"] == "fp32" else e
    if op == "norm":
        return {"bytes": 2 * n * e + 2 * d * w, "flops": 8 * n}
    return {"bytes": 3 * n * e + d * w + 8 * d, "flops": 17 * n}


# --------------------------------------------------------------------------
# 64-bit values, from the definitions
# --------------------------------------------------------------------------
_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_rows(x):
    """The values of x's rows in MXFP4, fp64 [rows, d], and the scales'
    exponents: nearest level by counting the borders between levels that a
    magnitude has passed."""
    rows, d = x.shape
    nb = (d + 31) // 32
    b = torch.zeros((rows, nb * 32), dtype=torch.float64, device=x.device)
    b[:, :d] = x.double()
    b = b.view(rows, nb, 32)
    top = b.abs().max(dim=-1, keepdim=True).values
    e = torch.floor(torch.log2(top)).clamp(min=-125.0) - 2.0
    # log2 may round up to a whole number just below a power of two
    e = torch.where(torch.exp2(e + 2.0) > top, e - 1.0, e).clamp(min=-127.0)
    scale = torch.exp2(e)
    level = torch.zeros(b.shape, dtype=torch.int64, device=x.device)
    a = b.abs() / scale
    for i in range(7):
        border = (_LEVELS[i] + _LEVELS[i + 1]) / 2.0
        # a tie goes to the even one of codes i and i + 1
        level += (a > border) if i % 2 == 0 else (a >= border)
    v = torch.tensor(_LEVELS, dtype=torch.float64, device=x.device)[level] * scale
    return (torch.sign(b) * v).view(rows, -1)[:, :d], e.squeeze(-1)


def _exact_codes(codes, scales):
    table = torch.tensor(_LEVELS + [-v for v in _LEVELS], dtype=torch.float64, device=codes.device)
    rows = codes.shape[0]
    v = torch.empty((rows, codes.shape[1], 2), dtype=torch.float64, device=codes.device)
    v[..., 0] = table[(codes % 16).long()]
    v[..., 1] = table[(codes // 16).long()]
    return (v.view(rows, -1, 32) * torch.exp2(scales.double() - 127.0)[..., None]).view(rows, -1)


def exact(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        x = d["x"].transpose(0, 1).contiguous() if case["columns"] else d["x"]
        v, e = _exact_rows(x)
        return [v, (e + 127.0).to(torch.uint8)]
    if op == "linear":
        w = _exact_codes(d["w_codes"], d["w_scales"])[:, :case["K"]]
        x = _exact_rows(d["x"])[0] if case["input"] == "values" else \
            _exact_codes(d["codes"], d["scales"])[:, :case["K"]]
        y = torch.matmul(x, w.t().contiguous())
        return y if d["bias"] is None else y + d["bias"].double()[None, :]
    if op == "back":
        up, up_t = _exact_rows(d["dout"])[0], _exact_rows(d["dout"].t().contiguous())[0]
        w_t, x_t = _exact_rows(d["weight"].t().contiguous())[0], _exact_rows(d["x"].t().contiguous())[0]
        return [torch.matmul(up, w_t.t().contiguous()), torch.matmul(up_t, x_t.t().contiguous()),
                torch.sum(d["dout"].double(), dim=0)]
    x, w = d["x"].double(), d["weight"].double()
    n = x.shape[1]
    mean = torch.sum(x, dim=1, keepdim=True) / n
    dev = torch.sqrt(torch.sum((x - mean) ** 2, dim=1, keepdim=True) / n + _EPS)
    z = (x - mean) / dev
    if op == "norm":
        return z * w[None, :] + d["bias"].double()[None, :]
    up = d["dout"].double()
    t = up * w[None, :]
    dx = (n * t - torch.sum(t, dim=1, keepdim=True) - z * torch.sum(t * z, dim=1, keepdim=True)) / (n * dev)
    return [dx, torch.sum(up * z, dim=0), torch.sum(up, dim=0)]
