"""GPU parity of the passes over heads: rotary positions and the paged append
bit for bit (every rounding is defined, given the table), the norms and their
gradients within the oracle's derived bounds."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer
from tests.gpu_util import TORCH_DT, assert_bits_equal, bits, case, dev, to_dev, torch

pytestmark = pytest.mark.gpu

DT = ["fp32", "fp16", "bf16"]
LAYOUTS = ["half", "interleaved"]


def tdt(t):
    return getattr(torch(), TORCH_DT[t])


def make(rng, shape, t, scale=1.0):
    b = layer.round_to((rng.standard_normal(shape) * scale).astype(np.float32), t)
    return b, layer.values(b, t)


def upload(b, t):
    d = torch().from_numpy(np.ascontiguousarray(b).view({2: np.int16, 4: np.int32}[b.dtype.itemsize])).to(dev())
    return d.view(tdt(t)).reshape(b.shape)


def table_of(rot, max_pos, **kw):
    f, amp = kb.rope_frequencies(rot, **kw)
    t = kb.rope_table(f, max_pos, amplitude=amp)
    return t, t.cpu().numpy()


def assert_close(got_bits, t, want, bound, what):
    """|got - want| <= bound, plus one rounding to the type."""
    got = layer.values(got_bits, t).astype(np.float64)
    rel, tiny = layer.half_ulp(t)
    lim = bound + rel * (np.abs(want) + bound) + tiny
    bad = np.argwhere(~(np.abs(got - want) <= lim))
    assert bad.size == 0, f"{what}: {len(bad)} of {want.size} outside, first {bad[:3].tolist()}"


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 250])
@pytest.mark.parametrize("kw", [{}, {"scaling": "linear", "factor": 3.0}, {"scaling": "ntk", "factor": 8.0},
                                {"scaling": "yarn", "factor": 4.0, "original_length": 500}])
def test_table(rot, kw):
    max_pos = 2003
    case(f"rope table rot={rot} {kw}")
    _, got = table_of(rot, max_pos, **kw)
    f, amp = layer.frequencies(rot, **kw)
    ang = np.arange(max_pos)[:, None] * f
    want = np.concatenate([amp * np.cos(ang), amp * np.sin(ang)], 1)
    # fp64 inside: angles within 2003 * 2^-45, then one fp32 rounding
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1e-9).all()


def test_table_far_positions():
    # at a million the angle still has 30 bits after the point
    case("rope table far")
    f, _ = kb.rope_frequencies(8)
    t = kb.rope_table(f, 1 << 20).cpu().numpy()
    want = np.cos(np.arange(1 << 20, dtype=np.float64)[:, None] * f)
    assert (np.abs(t[:, :4] - want) <= 2.0 ** -24 + 1e-9).all()


HEADS = [(1, 1, 2, 2), (3, 2, 3, 2), (5, 3, 16, 16), (4, 5, 64, 64), (7, 4, 64, 32), (2, 3, 80, 80), (6, 2, 96, 24),
         (33, 8, 128, 128), (9, 40, 128, 64), (3, 1, 192, 192), (5, 2, 256, 64), (2, 2, 100, 50), (3, 2, 72, 40),
         (2, 1, 1024, 1024), (2, 2, 1024, 512), (3, 1, 1001, 500), (300, 2, 64, 64)]


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,rot", HEADS)
def test_rope(t, layout, T, H, D, rot):
    case(f"rope {t} {layout} T={T} H={H} D={D} rot={rot}")
    rng = np.random.default_rng(T + H + D + rot)
    b, x = make(rng, (T, H, D), t)
    table, tab = table_of(rot, 1000)
    pos = rng.integers(0, 1000, T)
    for inverse, dt in ((False, np.int64), (True, np.int32)):
        got = kb.rope(upload(b, t), to_dev(pos.astype(dt)), table, layout=layout, inverse=inverse)
        want = layer.round_to(layer.rotate(x, pos, tab, layout, inverse), t)
        assert_bits_equal(bits(got), want, f"inverse={inverse}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_rope_strides_batches_and_in_place(t, layout):
    rng = np.random.default_rng(3)
    B, T, H, D, rot = 3, 7, 4, 64, 32
    table, tab = table_of(rot, 64)
    pos = rng.integers(0, 64, (B, T))
    b, x = make(rng, (B, T, H, D), t)
    want = layer.round_to(layer.rotate(x, pos, tab, layout), t)
    P = to_dev(pos)
    full = upload(b, t)
    views = {"contiguous": full.clone(),
             "head-major": full.transpose(1, 2).contiguous().transpose(1, 2),
             "token-first": full.transpose(0, 1).contiguous().transpose(0, 1)}
    wide = torch().full((B, T, H + 3, D + 5), 9.0, dtype=tdt(t), device=dev())  # odd strides: element by element
    wide[:, :, 1:H + 1, 3:D + 3] = full
    views["odd strides"] = wide[:, :, 1:H + 1, 3:D + 3]
    for name, v in views.items():
        case(f"rope {t} {layout} {name}")
        assert_bits_equal(bits(kb.rope(v, P, table, layout=layout).contiguous()), want, name)
        kb.rope(v, P, table, layout=layout, out=v)
        assert_bits_equal(bits(v.contiguous()), want, name + " in place")
    keep = torch().ones_like(wide, dtype=torch().bool)
    keep[:, :, 1:H + 1, 3:D + 3] = False
    assert (wide[keep] == 9.0).all()
    # a batch of single tokens, and single tokens of one batch
    assert_bits_equal(bits(kb.rope(full[:, 2:3], P[:, 2:3].contiguous(), table, layout=layout)), want[:, 2:3], "S=1")
    assert_bits_equal(bits(kb.rope(full[1], P[1], table, layout=layout)), want[1], "3-D")


def test_rope_special_values_and_positions():
    x = np.array([[[np.inf, 1.0, -np.inf, 2.0, np.inf, np.nan, -0.0, 5.0]]] * 4, np.float32)
    x[:, :, 5] = 3.0
    table, tab = table_of(4, 10)
    pos = np.array([0, 9, 10, -1])
    case("rope special")
    for layout in LAYOUTS:
        got = kb.rope(to_dev(x), to_dev(pos), table, layout=layout).cpu().numpy()
        want = layer.rotate(x, pos, tab, layout)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got[2:, 0, :4]).all()
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
        assert np.array_equal(got[:, :, 4:], x[:, :, 4:])  # not rotated: untouched, whatever the position


def test_rope_inverse_is_the_gradient():
    # <R x, g> = <x, R^T g>, in fp32 products summed in fp64: each side carries at most
    # 3 roundings an element
    rng = np.random.default_rng(6)
    b, x = make(rng, (50, 4, 96), "fp32")
    gb, g = make(rng, (50, 4, 96), "fp32")
    table, tab = table_of(64, 400, scaling="yarn", factor=4.0, original_length=100)
    pos = rng.integers(0, 400, 50)
    for layout in LAYOUTS:
        case(f"rope gradient {layout}")
        y = kb.rope(to_dev(x), to_dev(pos), table, layout=layout).double()
        dx = kb.rope(to_dev(g), to_dev(pos), table, layout=layout, inverse=True).double()
        left, right = (y * to_dev(g).double()).sum().item(), (dx * to_dev(x).double()).sum().item()
        mag = (np.abs(g) * layer.rotate_magnitude(x, pos, tab, layout)).sum()
        assert abs(left - right) <= 2 * layer.gamma(3) * mag


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,rot", HEADS)
def test_norm(t, layout, T, H, D, rot):
    case(f"norm {t} {layout} T={T} H={H} D={D} rot={rot}")
    rng = np.random.default_rng(T * 3 + H + D + rot)
    Hk = max(1, H // 3)
    qb, q = make(rng, (T, H, D), t, 3.0)
    kb_, k = make(rng, (T, Hk, D), t, 0.1)
    qb[0, 0] = 0  # a head of zeros: eps alone
    q = layer.values(qb, t)
    wt = "fp32" if (T + D) % 2 else t
    qwb, qw = make(rng, (D,), wt)
    kwb, kw = make(rng, (D,), wt)
    table, tab = table_of(rot, 500)
    pos = rng.integers(0, 500, T)
    eps = 1e-5
    qo, ko = kb.qk_norm_rope(upload(qb, t), upload(kb_, t), upload(qwb[None], wt)[0], upload(kwb[None], wt)[0],
                             to_dev(pos), table, eps=eps, layout=layout)
    eps32 = float(np.float32(eps))
    for got, x, w, what in ((qo, q, qw, "q"), (ko, k, kw, "k")):
        want, bound = layer.norm_rope(x, w, pos, tab, eps32, layout)
        assert_close(bits(got), t, want, bound, what)


@pytest.mark.parametrize("t", DT)
def test_norm_views_of_one_projection_in_place(t):
    rng = np.random.default_rng(10)
    B, T, Hq, Hk, D = 2, 5, 6, 2, 64
    b, x = make(rng, (B, T, (Hq + 2 * Hk) * D), t)
    qkv = upload(b, t)
    q = qkv[..., :Hq * D].view(B, T, Hq, D)
    k = qkv[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)
    qwb, qw = make(rng, (D,), t)
    kwb, kw = make(rng, (D,), t)
    table, tab = table_of(64, 50)
    pos = rng.integers(0, 50, (B, T))
    case(f"norm views {t}")
    kb.qk_norm_rope(q, k, upload(qwb[None], t)[0], upload(kwb[None], t)[0], to_dev(pos), table, q_out=q, k_out=k)
    eps = float(np.float32(1e-6))
    xq, xk = x[..., :Hq * D].reshape(B, T, Hq, D), x[..., Hq * D:(Hq + Hk) * D].reshape(B, T, Hk, D)
    for got, v, w in ((q, xq, qw), (k, xk, kw)):
        want, bound = layer.norm_rope(v, w, pos, tab, eps, "half")
        assert_close(bits(got.contiguous()), t, want, bound, "view")
    assert_bits_equal(bits(qkv[..., (Hq + Hk) * D:].contiguous()), b[..., (Hq + Hk) * D:], "v untouched")


def test_norm_not_finite():
    x = np.ones((4, 1, 32), np.float32)
    x[1, 0, 3] = np.nan
    x[2, 0, 4] = np.inf
    x[3] = 1e30  # the squares overflow: the norm is infinite, as in any fp32 evaluation
    table, tab = table_of(32, 8)
    case("norm not finite")
    one = torch().ones(32, device=dev())
    q, k = kb.qk_norm_rope(to_dev(x), to_dev(x), one, one, to_dev(np.arange(4)), table)
    q = q.cpu().numpy()
    assert np.isfinite(q[0]).all() and np.isnan(q[1]).all() and np.isnan(q[2, 0, 4]) and (q[3] == 0).all()
    assert np.array_equal(np.isnan(q), np.isnan(k.cpu().numpy()))


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,rot", [h for h in HEADS if h[0] < 300] + [(2000, 3, 64, 64), (5000, 1, 128, 32)])
def test_norm_gradient(t, layout, T, H, D, rot):
    case(f"norm gradient {t} {layout} T={T} H={H} D={D} rot={rot}")
    rng = np.random.default_rng(T * 5 + H + D + rot)
    Hk = max(1, H // 4)
    wt = "fp32" if (T + D) % 2 else t
    table, tab = table_of(rot, 500)
    pos = rng.integers(0, 500, T)
    d = {}
    for n, h in (("q", H), ("k", Hk)):
        d[n] = make(rng, (T, h, D), t, 2.0), make(rng, (T, h, D), t), make(rng, (D,), wt)
    (qb, q), (gqb, gq), (qwb, qw) = d["q"]
    (kb_, k), (gkb, gk), (kwb, kw) = d["k"]
    args = (upload(gqb, t), upload(gkb, t), upload(qb, t), upload(kb_, t), upload(qwb[None], wt)[0],
            upload(kwb[None], wt)[0], to_dev(pos), table)
    dq, dk, dqw, dkw = kb.qk_norm_rope_backward(*args, eps=1e-5, layout=layout)
    eps = float(np.float32(1e-5))
    for gx, gw, g, x, w, what in ((dq, dqw, gq, q, qw, "q"), (dk, dkw, gk, k, kw, "k")):
        dx, dxb, dw, dwb = layer.norm_rope_back(g, x, w, pos, tab, eps, layout)
        assert_close(bits(gx), t, dx, dxb, "d" + what)
        assert_close(bits(gw), "fp32", dw, dwb, f"d{what}_weight")
    again = kb.qk_norm_rope_backward(*args, eps=1e-5, layout=layout, dq=args[0], dk=args[1])  # over the gradients
    for a, b in zip(again, (dq, dk, dqw, dkw)):
        assert_bits_equal(bits(a), bits(b), "the same bits every time")


def test_norm_gradient_batches_and_no_tokens():
    rng = np.random.default_rng(12)
    B, T, H, D = 3, 5, 4, 64
    table, tab = table_of(64, 50)
    pos = rng.integers(0, 50, (B, T))
    (xb, x), (gb, g), (wb, w) = make(rng, (B, T, H, D), "bf16"), make(rng, (B, T, H, D), "bf16"), make(rng, (D,), "bf16")
    X = upload(xb, "bf16").transpose(1, 2).contiguous().transpose(1, 2)
    G, W = upload(gb, "bf16"), upload(wb[None], "bf16")[0]
    case("norm gradient batches")
    dq, dk, dqw, dkw = kb.qk_norm_rope_backward(G, G[:, :, :1], X, X[:, :, :1], W, W, to_dev(pos), table)
    eps = float(np.float32(1e-6))
    for gx, gw, gg, xx in ((dq, dqw, g, x), (dk, dkw, g[:, :, :1], x[:, :, :1])):
        dx, dxb, dw, dwb = layer.norm_rope_back(gg, xx, w, pos, tab, eps, "half")
        assert_close(bits(gx), "bf16", dx, dxb, "dx")
        assert_close(bits(gw), "fp32", dw, dwb, "dw")
    case("norm gradient no tokens")
    e = G[:, :0]
    out = kb.qk_norm_rope_backward(e, e, e, e, W, W, to_dev(pos)[:, :0].contiguous(), table)
    assert out[0].numel() == 0 and not out[2].any() and not out[3].any()


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,Dv,rot,page,order", [(1, 1, 64, 64, 64, 1, "token"), (5, 2, 128, 128, 128, 16, "token"),
                                                     (40, 3, 128, 64, 64, 16, "head"), (33, 8, 80, 80, 80, 32, "head"),
                                                     (7, 2, 50, 30, 20, 5, "token"), (9, 1, 96, 96, 0, 64, "token"),
                                                     (130, 5, 64, 128, 64, 16, "head"), (3, 2, 1001, 8, 1000, 4, "head")])
def test_append(t, layout, T, H, D, Dv, rot, page, order):
    case(f"append {t} {layout} T={T} H={H} D={D} Dv={Dv} rot={rot} page={page} {order}")
    rng = np.random.default_rng(T + H + D + page)
    pages = -(-T // page) + 2
    (kb_, k), (vb, v) = make(rng, (T, H, D), t), make(rng, (T, H, Dv), t)
    kcb, _ = make(rng, (pages, page, H, D), t)
    vcb, _ = make(rng, (pages, page, H, Dv), t)
    slots = rng.permutation(pages * page)[:T]
    if T > 4:
        slots[1], slots[2], slots[3] = -1, pages * page, -(1 << 31)
    pos = rng.integers(0, 300, T)
    kw, rows = {}, kb_
    if rot:
        table, tab = table_of(rot, 300)
        kw = {"positions": to_dev(pos), "table": table, "layout": layout}
        rows = layer.round_to(layer.rotate(k, pos, tab, layout), t)
    caches = [upload(c, t) for c in (kcb, vcb)]
    if order == "head":
        caches = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in caches]
    slot_t = np.int32 if T % 2 else np.int64
    kb.append_kv_paged(upload(kb_, t), upload(vb, t), to_dev(slots.astype(slot_t)), *caches, **kw)
    assert_bits_equal(bits(caches[0].contiguous()), layer.append(kcb, rows, slots), "k_cache")
    assert_bits_equal(bits(caches[1].contiguous()), layer.append(vcb, vb, slots), "v_cache")


def test_append_far_into_a_large_cache():
    # the last page's offset passes 2^32 bytes
    t = torch()
    page, H, D = 64, 8, 128
    pages = (1 << 32) // (page * H * D * 2) + 2
    k_cache = t.zeros(pages, page, H, D, dtype=t.bfloat16, device=dev())
    v_cache = t.zeros(1, page, H, D, dtype=t.bfloat16, device=dev()).expand(pages, page, H, D)  # one page for all
    k = t.randn(2, H, D, dtype=t.bfloat16, device=dev())
    slots = t.tensor([pages * page - 1, 5], device=dev())
    case("append far")
    kb.append_kv_paged(k, k, slots, k_cache, v_cache)
    assert t.equal(k_cache[-1, -1], k[0]) and t.equal(k_cache[0, 5], k[1])
    assert int((k_cache[-1] != 0).any(-1).any(-1).sum()) == 1


def test_refusals():
    t = torch()
    x = t.zeros(4, 2, 64, device=dev())
    table, _ = table_of(64, 16)
    pos = t.zeros(4, dtype=t.int64, device=dev())
    w = t.ones(64, device=dev())
    cache = t.zeros(3, 4, 2, 64, device=dev())
    for fn, match in ((lambda: kb.rope(x, pos[:3], table), "positions"),
                      (lambda: kb.rope(x, pos.float(), table), "positions"),
                      (lambda: kb.rope(x, pos.cpu(), table), "positions"),
                      (lambda: kb.rope(x, pos, table.double()), "table"),
                      (lambda: kb.rope(x[..., :32], pos, table), "rotates"),
                      (lambda: kb.rope(x, pos, table, layout="other"), "layout"),
                      (lambda: kb.rope(x.transpose(1, 2), pos, table), "contiguous"),
                      (lambda: kb.rope(x, pos, table, out=x[:3]), "out"),
                      (lambda: kb.qk_norm_rope(x, x[:3], w, w, pos, table), "heads only"),
                      (lambda: kb.qk_norm_rope(x, x, w[:32], w, pos, table), "q_weight"),
                      (lambda: kb.qk_norm_rope(x, x, w, w.half(), pos, table), "k_weight"),
                      (lambda: kb.qk_norm_rope(x, x.half(), w, w, pos, table), "k: element type"),
                      (lambda: kb.qk_norm_rope_backward(x[:3], x, x, x, w, w, pos, table), "dq_out"),
                      (lambda: kb.append_kv_paged(x, x[:3], pos, cache, cache), "differ"),
                      (lambda: kb.append_kv_paged(x, x, pos, cache[:, :, :1], cache), "k_cache"),
                      (lambda: kb.append_kv_paged(x, x, pos, cache, cache[:2]), "v_cache"),
                      (lambda: kb.append_kv_paged(x, x, pos[:2], cache, cache), "slots"),
                      (lambda: kb.append_kv_paged(x, x, pos, cache, cache, positions=pos), "both")):
        with pytest.raises((ValueError, TypeError), match=match):
            fn()
    with pytest.raises(kb.KbitError):
        kb.qk_norm_rope(x, x, w, w, pos, table, eps=-1.0)


def test_graph_of_the_chain():
    # int8 projection -> norms with rotation -> append, captured once
    t = torch()
    rng = np.random.default_rng(20)
    T, Hq, Hk, D, K = 6, 4, 2, 64, 256
    X = upload(make(rng, (T, K), "bf16")[0], "bf16")
    W, sw = kb.quantize_rows_int8(upload(make(rng, ((Hq + 2 * Hk) * D, K), "bf16")[0], "bf16"))
    qw, kw = (upload(make(rng, (1, D), "bf16")[0], "bf16")[0] for _ in range(2))
    table, _ = table_of(64, 100)
    pos, slots = to_dev(rng.integers(0, 100, T)), to_dev(rng.permutation(64)[:T])
    kc, vc = (t.zeros(4, 16, Hk, D, dtype=t.bfloat16, device=dev()) for _ in range(2))
    qkv = t.empty(T, (Hq + 2 * Hk) * D, dtype=t.bfloat16, device=dev())
    q, k, v = (qkv[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))

    def step():
        kb.linear_int8_dynamic(X, W, sw, out=qkv)
        kb.qk_norm_rope(q, k, qw, kw, pos, table, q_out=q, k_out=k)
        kb.append_kv_paged(k, v, slots, kc, vc)

    case("graph of the chain")
    step()
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        step()
    for i in range(4):
        X.copy_(X.roll(1, 0))
        step()
        want = [c.clone() for c in (qkv, kc, vc)]
        qkv.zero_(), kc.zero_(), vc.zero_()
        g.replay()
        t.cuda.synchronize()
        for a, b, what in zip((qkv, kc, vc), want, ("qkv", "k_cache", "v_cache")):
            assert_bits_equal(bits(a), bits(b), f"{what}, replay {i}")
