"""moe_expert_matmul and its gradients against the 64-bit formulas: every activation, ragged and empty
experts, padded and capacity layouts, odd sizes, rows that hold no token (NaN on entry, untouched on
return), captured graphs and streams.

Tolerances.  u = 2^-8 is half a bf16 step, relative.  A sum of K products of bf16 values (exact in
fp32) takes K additions, each off by at most 2^-23 of the terms' magnitude (2^-24 rounded to nearest,
2^-23 if the unit truncates): (K + 2) 2^-23 sum|x||w|.  The activations change by at most 1.13 times
their argument's error; their fp32 evaluation (exp, erf, a quotient) is off by at most 2^-18 relative
for |z| < 64.  Each output is rounded to bf16 once.  grad_pre is rounded to bf16 before the products
read it, which adds u sum|d||w| at most.
"""
import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
SENTINEL = 7.0


def _mod():
    import combine_moe_route_07_b200 as m
    return m


def _layout(m, T, E, k, align=1, cap=0, seed=0, only=None, home=None):
    """Shape, workspace, layout and the rows' 64-bit segments for random ids (`only`: the experts
    tokens may choose)."""
    g = torch.Generator().manual_seed(seed)
    key = torch.rand(T, E, generator=g)
    if only is not None:
        mask = torch.full((E,), -10.0)
        mask[list(only)] = 0.0
        key = key + mask
    ids = torch.topk(key, k, dim=1).indices.to(torch.int32).cuda()
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1 if home is None else E,
                       capacity=cap, align=align)
    ws = m.Workspace(shape)
    lay = m.moe_layout(shape, ids, ws=ws) if home is None else \
        m.moe_layout_remote_first(shape, ids, home, ws=ws)[0]
    segs = ref.segments(lay.counts.cpu(), lay.expert_off.cpu(), cap, E)
    held = torch.zeros(shape.rows, dtype=torch.bool)
    for r in segs:
        held[r] = True
    return shape, ws, lay, segs, held


def _rows(n, cols, held, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(n, cols, generator=g) * scale).to(torch.bfloat16)
    v[~held] = float("nan")
    return v


def _weights(E, W, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(E, W, K, generator=g) / K ** 0.5).to(torch.bfloat16)


def _sum_tol(K, mag):
    return (K + 2) * 2.0 ** -23 * mag


def _check(got, want, tol, held, what):
    got = got.cpu()
    assert (got[~held] == SENTINEL).all(), f"{what}: a row without a token was written"
    d = (got[held].double() - want[held]).abs()
    assert torch.isfinite(got[held]).all(), what
    over = d - tol[held]
    assert (over <= 0).all(), f"{what}: worst {over.max().item():.3g} over, error {d.max().item():.3g}"


def _forward_case(T, E, k, K, F, name, bias, residual, pre, align=1, cap=0, only=None, home=None, seed=1):
    m = _mod()
    shape, ws, lay, segs, held = _layout(m, T, E, k, align, cap, seed, only, home)
    n = shape.rows
    W = 2 * F if name == "swiglu" else F
    x, w = _rows(n, K, held, seed + 1), _weights(E, W, K, seed + 2)
    b = torch.randn(E, W, generator=torch.Generator().manual_seed(seed + 3)) * 0.3 if bias else None
    res = _rows(n, F, held, seed + 4) if residual else None
    want, z, mag = ref.matmul(x, w, segs, b, name, res)
    out = torch.full((n, F), SENTINEL, dtype=torch.bfloat16, device="cuda")
    zb = torch.full((n, W), SENTINEL, dtype=torch.bfloat16, device="cuda") if pre else None
    m.moe_expert_matmul(shape, x.cuda(), w.cuda(), lay.counts, lay.expert_off, ws=ws,
                        bias=None if b is None else b.cuda(), act=name,
                        residual=None if res is None else res.cuda(), out=out, pre=zb)
    m.moe_check(ws)
    zt = _sum_tol(K, mag)
    if name == "swiglu":  # product of silu(gate) and up
        gate, up = z[:, :F], z[:, F:]
        s = (gate * torch.sigmoid(gate)).abs()
        t = 1.13 * zt[:, :F] * (up.abs() + zt[:, F:]) + s * zt[:, F:] + 2.0 ** -18 * s * up.abs()
    else:
        y = ref.act(z, name).abs()
        t = 1.13 * zt + 2.0 ** -18 * (y + z.abs() * (name != "none"))
    extra = 0 if res is None else 2.0 ** -24 * (want.abs() + res.double().nan_to_num().abs())
    _check(out, want, (t + extra) * (1 + U) + U * want.abs(), held, "out")
    if pre:
        _check(zb, z, zt * (1 + U) + U * z.abs(), held, "pre")


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("bias,residual,pre", [(False, False, False), (True, True, True)])
def test_activations_and_epilogue(name, bias, residual, pre):
    _forward_case(150, 8, 2, 192, 136, name, bias, residual, pre)


@pytest.mark.parametrize("T,E,k,K,F", [
    (1, 1, 1, 8, 8), (1, 4, 2, 64, 64), (2, 3, 1, 8, 264), (17, 2, 1, 72, 8), (15, 1, 1, 1000, 128),
    (16, 1, 1, 64, 128), (129, 1, 1, 64, 136), (255, 1, 1, 128, 256), (256, 1, 1, 128, 256),
    (257, 1, 1, 136, 248), (511, 2, 1, 520, 384), (1025, 3, 2, 256, 520), (600, 64, 6, 128, 72),
    (40, 1024, 4, 64, 16), (4200, 1, 1, 64, 40), (9000, 1024, 4, 16, 24), (2100, 512, 8, 24, 16),
    (700, 5, 3, 64, 1032), (64, 1, 1, 4104, 64),
])
@pytest.mark.parametrize("name", ["silu", "swiglu"])
def test_sizes(T, E, k, K, F, name):
    _forward_case(T, E, k, K, F, name, True, False, False)


@pytest.mark.parametrize("align,cap", [(16, 0), (128, 0), (3, 0), (1, 5), (1, 64)])
def test_padded_and_capacity_layouts(align, cap):
    _forward_case(300, 12, 3, 200, 144, "gelu", True, True, True, align, cap)


def test_experts_without_rows_and_remote_first_order():
    _forward_case(90, 16, 2, 128, 64, "swiglu", True, False, True, only=(3, 4, 11))
    _forward_case(90, 6, 2, 128, 64, "none", False, True, False, home=2, align=8)


def test_band_of_many_token_tiles():
    _forward_case(9001, 1, 1, 128, 392, "none", True, False, False)


def test_dense_call_and_residual_in_place():
    m = _mod()
    T, K, F = 333, 256, 256
    shape = m.MoeShape(tokens=T, hidden=8, experts=1, k=1, ranks=1)
    ws = m.Workspace(shape)
    held = torch.ones(T, dtype=torch.bool)
    x, w = _rows(T, K, held, 1), _weights(1, F, K, 2)
    want, z, mag = ref.matmul(x, w, [slice(0, T)], None, "relu", x)
    out = x.cuda()
    y = m.moe_expert_matmul(shape, x.cuda(), w.cuda(), ws=ws, act="relu", residual=out, out=out)
    assert y is out
    m.moe_check(ws)
    _check(out, want, (1.13 * _sum_tol(K, mag) + 2.0 ** -23 * (want.abs() + x.double().abs())) * (1 + U)
           + U * want.abs(), held, "out")


def test_nan_and_inf_stay_in_their_row():
    m = _mod()
    T, K, F = 40, 64, 128
    shape = m.MoeShape(tokens=T, hidden=8, experts=1, k=1, ranks=1)
    ws = m.Workspace(shape)
    x, w = _rows(T, K, torch.ones(T, dtype=torch.bool), 1), _weights(1, F, K, 2)
    clean = m.moe_expert_matmul(shape, x.cuda(), w.cuda(), ws=ws).cpu()
    x[7, 3], x[21, 5] = float("nan"), float("inf")
    got = m.moe_expert_matmul(shape, x.cuda(), w.cuda(), ws=ws).cpu()
    assert torch.isnan(got[7]).all() and not torch.isfinite(got[21]).any()
    keep = [i for i in range(T) if i not in (7, 21)]
    assert torch.equal(got[keep], clean[keep])


def _backward_case(T, E, k, K, F, name, align=1, cap=0, only=None, seed=5):
    m = _mod()
    shape, ws, lay, segs, held = _layout(m, T, E, k, align, cap, seed, only)
    n = shape.rows
    W = 2 * F if name == "swiglu" else F
    x, w = _rows(n, K, held, seed + 1), _weights(E, W, K, seed + 2)
    dy = _rows(n, F, held, seed + 3)
    z = _rows(n, W, held, seed + 4, 1.5)
    gx, gw, gb, gp, mx, mw, mb = ref.matmul_grads(dy, x, w, z, segs, name)
    full = lambda *s: torch.full(s, SENTINEL, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    got = m.moe_expert_matmul_backward(
        shape, dy.cuda(), x.cuda(), w.cuda(), lay.counts, lay.expert_off, ws=ws, act=name,
        pre=None if name == "none" else z.cuda(), grad_x=full(n, K),
        grad_pre=None if name == "none" else full(n, W), need_bias=True)
    m.moe_check(ws)
    rounded = 0.0 if name == "none" else U
    # the slope's fp32 evaluation: at most 2^-18 of the terms it is a sum of, which are below 4 |dy|
    # (swiglu: 4 |dy| times the other half)
    one = dy.double().nan_to_num().abs()
    if name == "swiglu":
        zz = z.double().nan_to_num().abs()
        slope = torch.cat([one * zz[:, F:], one * (1 + zz[:, :F])], 1) * 4 * 2.0 ** -18
    else:
        slope = one * 4 * 2.0 ** -18 * (name != "none")
    if name != "none":
        _check(got.grad_pre, gp, slope * (1 + U) + U * gp.abs(), held, "grad_pre")
    # magnitudes of what the products sum, with the slope's error pushed through them
    sx, sw = torch.zeros_like(gx), torch.zeros_like(gw)
    sb = torch.zeros_like(gb)
    for e, r in enumerate(segs):
        if r.stop > r.start:
            sx[r] = slope[r] @ w[e].double().abs()
            sw[e] = slope[r].T @ x[r].double().abs()
            sb[e] = slope[r].sum(0)
    most = max(max(r.stop - r.start for r in segs), 1)
    _check(got.grad_x, gx, (_sum_tol(W, mx) + rounded * mx + sx) * (1 + 2 * U) + U * gx.abs(), held, "grad_x")
    every = torch.ones(E, dtype=torch.bool)
    _check(got.grad_w, gw, (_sum_tol(most, mw) + rounded * mw + sw) * (1 + 2 * U) + U * gw.abs(), every, "grad_w")
    _check(got.grad_bias, gb, (most + 16) * 2.0 ** -24 * mb + sb * 1.001 + 2.0 ** -24 * gb.abs(), every, "grad_bias")


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "silu", "swiglu"])
def test_gradients(name):
    _backward_case(150, 8, 2, 192, 136, name)


@pytest.mark.parametrize("T,E,k,K,F", [
    (1, 1, 1, 8, 8), (1, 4, 2, 64, 64), (15, 1, 1, 264, 40), (16, 1, 1, 64, 128), (17, 2, 1, 72, 8),
    (64, 1, 1, 128, 128), (65, 1, 1, 520, 136), (300, 3, 2, 136, 264), (40, 128, 4, 64, 16),
    (1100, 2, 1, 72, 264), (3000, 1024, 4, 16, 24), (2100, 512, 8, 24, 16), (700, 5, 3, 648, 40),
])
def test_gradient_sizes(T, E, k, K, F):
    _backward_case(T, E, k, K, F, "swiglu")
    _backward_case(T, E, k, K, F, "none")


@pytest.mark.parametrize("align,cap", [(16, 0), (3, 0), (1, 5), (1, 64)])
def test_gradients_of_padded_and_capacity_layouts(align, cap):
    _backward_case(300, 12, 3, 200, 144, "gelu", align, cap)


def test_gradients_with_experts_without_rows():
    _backward_case(90, 16, 2, 128, 64, "swiglu", only=(3, 4, 11))


def test_gradients_agree_with_differences():
    """Central differences of the 64-bit forward at the same operands."""
    m = _mod()
    shape, ws, lay, segs, held = _layout(m, 12, 3, 2, seed=3)
    n, K, F, name = shape.rows, 16, 8, "swiglu"
    x, w, dy = _rows(n, K, held, 1), _weights(3, 2 * F, K, 2), _rows(n, F, held, 3)
    b = torch.zeros(3, 2 * F)
    zb = torch.empty(n, 2 * F, dtype=torch.bfloat16, device="cuda")
    m.moe_expert_matmul(shape, x.cuda(), w.cuda(), lay.counts, lay.expert_off, ws=ws, act=name, pre=zb)
    got = m.moe_expert_matmul_backward(shape, dy.cuda(), x.cuda(), w.cuda(), lay.counts, lay.expert_off,
                                       ws=ws, act=name, pre=zb, need_bias=True)
    h = 1e-4

    def loss(xx, ww, bb):
        return (ref.matmul(xx, ww, segs, bb, name)[0] * dy.double()).sum()

    xd, wd, bd = x.double(), w.double(), b.double()
    g = torch.Generator().manual_seed(9)
    for which, grad, base in ((0, got.grad_x, xd), (1, got.grad_w, wd), (2, got.grad_bias, bd)):
        norm = grad.double().norm().item()
        for _ in range(12):
            i = int(torch.randint(base.numel(), (1,), generator=g))
            step = torch.zeros(base.numel(), dtype=torch.float64)
            step[i] = h
            step = step.reshape(base.shape)
            args = [xd, wd, bd]
            up, dn = list(args), list(args)
            up[which], dn[which] = base + step, base - step
            want = (loss(*up) - loss(*dn)).item() / (2 * h)
            # pre and grad_pre are rounded to bf16 (2^-8 of each of the at most 24 terms, whose
            # magnitudes the gradient's norm bounds), differences to h^2
            assert abs(grad.reshape(-1)[i].item() - want) <= 4 * U * (abs(want) + norm) + 1e-6


def test_single_gradients_and_dense_backward():
    m = _mod()
    T, K, F = 70, 64, 72
    shape = m.MoeShape(tokens=T, hidden=8, experts=1, k=1, ranks=1)
    ws = m.Workspace(shape)
    held = torch.ones(T, dtype=torch.bool)
    x, w, dy = _rows(T, K, held, 1).cuda(), _weights(1, F, K, 2).cuda(), _rows(T, F, held, 3).cuda()
    all3 = m.moe_expert_matmul_backward(shape, dy, x, w, ws=ws, need_bias=True)
    for name in ("x", "w", "bias"):
        need = {f"need_{q}": q == name for q in ("x", "w", "bias")}
        one = m.moe_expert_matmul_backward(shape, dy, x, w, ws=ws, **need)
        for q in ("x", "w", "bias"):
            a, b = getattr(one, f"grad_{q}"), getattr(all3, f"grad_{q}")
            assert (torch.equal(a, b) if q == name else a is None)
    m.moe_check(ws)


def test_no_tokens():
    m = _mod()
    shape = m.MoeShape(tokens=0, hidden=8, experts=4, k=2, ranks=1)
    ws = m.Workspace(shape)
    w = torch.randn(4, 16, 8, device="cuda").to(torch.bfloat16)
    z = torch.zeros(4, dtype=torch.int32, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    assert m.moe_expert_matmul(shape, x, w, z, off, ws=ws).shape == (0, 16)
    dy = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    g = m.moe_expert_matmul_backward(shape, dy, x, w, z, off, ws=ws, need_bias=True)
    assert (g.grad_w == 0).all() and (g.grad_bias == 0).all() and g.grad_x.shape == (0, 8)


def test_results_do_not_change_between_calls_and_graph_replays():
    m = _mod()
    shape, ws, lay, segs, held = _layout(m, 700, 8, 2, seed=11)
    n, K, F = shape.rows, 320, 264
    x, w, dy = _rows(n, K, held, 1).cuda(), _weights(8, 2 * F, K, 2).cuda(), _rows(n, F, held, 3).cuda()
    out = torch.zeros(n, F, dtype=torch.bfloat16, device="cuda")
    pre = torch.zeros(n, 2 * F, dtype=torch.bfloat16, device="cuda")
    bufs = dict(grad_pre=torch.zeros_like(pre), grad_x=torch.zeros(n, K, dtype=torch.bfloat16, device="cuda"),
                grad_w=torch.zeros_like(w), grad_bias=torch.zeros(8, 2 * F, device="cuda"))

    def step():
        m.moe_expert_matmul(shape, x, w, lay.counts, lay.expert_off, ws=ws, act="swiglu", out=out, pre=pre)
        m.moe_expert_matmul_backward(shape, dy, x, w, lay.counts, lay.expert_off, ws=ws, act="swiglu",
                                     pre=pre, **bufs)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, pre, *bufs.values())]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    for _ in range(3):
        for t in (out, pre, *bufs.values()):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, v in zip((out, pre, *bufs.values()), want):
            assert torch.equal(t, v)
    m.moe_check(ws)


def test_two_streams_at_once():
    m = _mod()
    T, K, F = 900, 512, 640
    shape = m.MoeShape(tokens=T, hidden=8, experts=1, k=1, ranks=1)
    held = torch.ones(T, dtype=torch.bool)
    w = _weights(1, F, K, 2).cuda()
    xs = [_rows(T, K, held, i).cuda() for i in range(2)]
    wss = [m.Workspace(shape) for _ in range(2)]
    want = [m.moe_expert_matmul(shape, x, w, ws=s) for x, s in zip(xs, wss)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(m.moe_expert_matmul(shape, xs[i], w, ws=wss[i]))
    torch.cuda.synchronize()
    for i in range(2):
        m.moe_check(wss[i])
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_bad_segments_are_reported_and_skipped():
    m = _mod()
    from combine_moe_route_07_b200 import _binding
    shape, ws, lay, segs, held = _layout(m, 60, 4, 1, seed=2)
    n, K, F = shape.rows, 64, 64
    x, w = _rows(n, K, held, 1).cuda(), _weights(4, F, K, 2).cuda()
    want = m.moe_expert_matmul(shape, x, w, lay.counts, lay.expert_off, ws=ws).cpu()
    for change, detail in ((("off", 2, -5), 2), (("off", 1, n), 1), (("counts", 3, -1), 3),
                           (("counts", 0, n + 1), 0)):
        off, counts = lay.expert_off.clone(), lay.counts.clone()
        (off if change[0] == "off" else counts)[change[1]] = change[2]
        out = torch.full((n, F), SENTINEL, dtype=torch.bfloat16, device="cuda")
        m.moe_expert_matmul(shape, x, w, counts, off, ws=ws, out=out)
        assert m.moe_get_device_error(ws) == (_binding.MOE_ERR_DEVICE_RANGE, detail)
        out = out.cpu()
        for e, r in enumerate(segs):
            assert torch.equal(out[r], want[r]) if e != change[1] else (out[r] == SENTINEL).all()
    # segments that overlap hold more rows than there are assignments
    off, counts = torch.zeros_like(lay.expert_off), torch.full_like(lay.counts, n)
    out = torch.full((n, F), SENTINEL, dtype=torch.bfloat16, device="cuda")
    m.moe_expert_matmul(shape, x, w, counts, off, ws=ws, out=out)
    assert m.moe_get_device_error(ws) == (_binding.MOE_ERR_DEVICE_RANGE, 4)
    assert (out == SENTINEL).all()
    g = m.moe_expert_matmul_backward(shape, want.cuda(), x, w, counts, off, ws=ws, need_bias=True,
                                     need_w=False)
    assert m.moe_get_device_error(ws) == (_binding.MOE_ERR_DEVICE_RANGE, 4)
    assert (g.grad_bias == 0).all()


def test_offsets_past_32_bits():
    """More than 2^31 elements in a matrix: the last rows are where they belong."""
    m = _mod()
    T, K, F, last = 70001, 8, 32768, 70001 - 130
    assert T * F > 1 << 31
    shape = m.MoeShape(tokens=T, hidden=8, experts=1, k=1, ranks=1)
    ws = m.Workspace(shape)
    x, w = torch.randn(T, K, device="cuda").to(torch.bfloat16), _weights(1, F, K, 2).cuda()
    out = m.moe_expert_matmul(shape, x, w, ws=ws)
    m.moe_check(ws)
    for r in (slice(0, 64), slice(32768, 32800), slice(last, T)):
        want, z, mag = ref.matmul(x[r].cpu(), w.cpu(), [slice(0, r.stop - r.start)])
        _check(out[r], want, _sum_tol(K, mag) * (1 + U) + U * want.abs(),
               torch.ones(r.stop - r.start, dtype=torch.bool), "out")
    # rows and weights gradients over the same matrix
    g = m.moe_expert_matmul_backward(shape, out, x, w, ws=ws, need_bias=True)
    m.moe_check(ws)
    d = out[last:].double().cpu()
    gx = d @ w[0].double().cpu()
    mx = d.abs() @ w[0].double().cpu().abs()
    _check(g.grad_x[last:], gx, _sum_tol(F, mx) * (1 + U) + U * gx.abs(),
           torch.ones(T - last, dtype=torch.bool), "grad_x")
    cols = slice(F - 256, F)
    dc = out[:, cols].double()
    gw, mw = dc.T @ x.double(), dc.abs().T @ x.double().abs()
    _check(g.grad_w[0, cols], gw.cpu(), (_sum_tol(T, mw) * (1 + U) + U * gw.abs()).cpu(),
           torch.ones(256, dtype=torch.bool), "grad_w")
    _check(g.grad_bias[:, cols], dc.sum(0)[None].cpu(), ((T + 16) * 2.0 ** -24 * dc.abs().sum(0))[None].cpu(),
           torch.ones(1, dtype=torch.bool), "grad_bias")


def test_wrong_tensors_are_refused():
    m = _mod()
    shape, ws, lay, segs, held = _layout(m, 10, 4, 1, seed=2)
    n = shape.rows
    x, w = _rows(n, 64, held, 1).cuda(), _weights(4, 16, 64, 2).cuda()
    call = lambda **kw: m.moe_expert_matmul(  # noqa: E731
        shape, kw.pop("x", x), kw.pop("w", w), kw.pop("counts", lay.counts), kw.pop("off", lay.expert_off),
        ws=ws, **kw)
    for kw in (dict(x=x.float()), dict(x=x[:, :32]), dict(x=x.cpu()), dict(w=w[:3]), dict(w=w.transpose(1, 2)),
               dict(act="tanh"), dict(counts=lay.counts.long()), dict(bias=torch.zeros(4, 8, device="cuda")),
               dict(residual=x), dict(out=x), dict(off=lay.expert_off[:4])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(m.MoeError):  # features that are no multiple of 8
        call(w=w[:, :12].contiguous())
    with pytest.raises(m.MoeError):  # only one of the two
        call(counts=None)
    with pytest.raises(m.MoeError):  # four experts need a layout
        call(counts=None, off=None)
    with pytest.raises(m.MoeError):  # an activation's gradient needs the pre-activations
        m.moe_expert_matmul_backward(shape, _rows(n, 16, held, 3).cuda(), x, w, lay.counts, lay.expert_off,
                                     ws=ws, act="gelu")


def _gelu_tail_tol(z):
    """Relative error of Phi(-|z|) in fp32: the scaled tail's polynomial (2^-20.7 with its roundings),
    the exponential (2^-22) and three products (2^-24 each): 17 steps of 2^-24; the exponent z^2 / 2 takes
    two roundings and a constant off by 0.23 of one, each 2^-24 of it: 1.12 z^2 steps."""
    return (18.0 + 1.2 * z * z) * 2.0 ** -24


def test_gelu_of_far_negative_values():
    """The tail is held relative to itself: at z = -10 the result is 1e-22, and bf16 shows 2^-8 of that."""
    m = _mod()
    F = 4096
    z = torch.cat([torch.linspace(-13.0, -3.0, F - 1024), torch.linspace(-3.0, 12.0, 1024)])
    shape = m.MoeShape(tokens=3, hidden=8, experts=1, k=1, ranks=1)
    x = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, F, 8, dtype=torch.bfloat16, device="cuda")
    got = m.moe_expert_matmul(shape, x, w, ws=m.Workspace(shape), act="gelu", bias=z[None].cuda())
    zd = z.double()
    want = 0.5 * zd * torch.erfc(-zd / 2.0 ** 0.5)
    tol = (U + _gelu_tail_tol(zd) * (1 + U)) * want.abs()
    for row in got.cpu().double():
        assert ((row - want).abs() <= tol).all()


def test_gelu_slope_of_far_negative_values():
    """The bias gradient of one row is the slope in fp32, before any rounding to bf16."""
    m = _mod()
    F = 4096
    z = torch.cat([torch.linspace(-13.0, -3.0, F - 1024), torch.linspace(-3.0, 12.0, 1024)]).to(torch.bfloat16)
    shape = m.MoeShape(tokens=1, hidden=8, experts=1, k=1, ranks=1)
    x = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, F, 8, dtype=torch.bfloat16, device="cuda")
    got = m.moe_expert_matmul_backward(shape, torch.ones(1, F, dtype=torch.bfloat16, device="cuda"), x, w,
                                       ws=m.Workspace(shape), act="gelu", pre=z[None].cuda(), need_x=False,
                                       need_bias=True)
    zd = z.double()
    phi, Phi = torch.exp(-0.5 * zd * zd) / (2.0 * torch.pi) ** 0.5, 0.5 * torch.erfc(-zd / 2.0 ** 0.5)
    want, mag = Phi + zd * phi, Phi + zd.abs() * phi
    err = (got.grad_bias[0].cpu().double() - want).abs()
    assert (err <= _gelu_tail_tol(zd) * mag).all()
    off = (got.grad_pre[0].cpu().double() - want).abs()
    assert (off <= U * want.abs() + (1 + U) * _gelu_tail_tol(zd) * mag).all()
