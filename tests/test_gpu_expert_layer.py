"""The combine's gradients against the formulas, and a whole expert layer as a training step uses it:
scored route, layout, dispatch, the two expert products, combine, and the gradients back to the input,
the logits and every weight, against automatic differentiation in 64 bits."""
import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _mod():
    import combine_moe_route_07_b200 as m
    return m


def _randn(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


@pytest.mark.parametrize("T,H,E,k,cap,align", [
    (1, 8, 1, 1, 0, 1), (3, 24, 4, 2, 0, 1), (130, 1032, 16, 4, 0, 1), (257, 264, 32, 8, 0, 16),
    (64, 4096, 64, 8, 0, 1), (100, 7168, 16, 3, 9, 1), (33, 520, 64, 10, 0, 1), (20, 256, 64, 32, 0, 1),
    (40, 2048, 8, 8, 3, 1), (3000, 512, 16, 2, 0, 1), (9, 32768, 8, 2, 0, 1), (700, 136, 40, 17, 40, 1),
])
def test_combine_backward(T, H, E, k, cap, align):
    m = _mod()
    shape = m.MoeShape(tokens=T, hidden=H, experts=E, k=k, ranks=1, capacity=cap, align=align)
    ws = m.Workspace(shape)
    ids = torch.topk(_randn(T, E, seed=1), k, dim=1).indices.int().cuda()
    lay = m.moe_layout(shape, ids, ws=ws)
    dst = lay.dst_pos.cpu().long()
    n = shape.rows
    held = torch.zeros(n, dtype=torch.bool)
    held[dst[dst >= 0]] = True
    y, dout = _randn(n, H, seed=2).to(torch.bfloat16), _randn(T, H, seed=3).to(torch.bfloat16)
    y[~held] = float("nan")
    gates = torch.softmax(_randn(T, k, seed=4), 1)
    grad_y = torch.full((n, H), 7.0, dtype=torch.bfloat16, device="cuda")
    gates_in = gates.clone()
    gates_in[dst < 0] = float("nan")  # a dropped slot's gate plays no part
    gy, gg = m.moe_combine_backward(shape, dout.cuda(), y.cuda(), lay.dst_pos, gates_in.cuda(), ws=ws,
                                    grad_y=grad_y)
    m.moe_check(ws)
    gy, gg = gy.cpu(), gg.cpu()
    t, j = torch.nonzero(dst >= 0, as_tuple=True)
    want = torch.zeros(n, H, dtype=torch.float64)
    want[dst[t, j]] = gates[t, j].double()[:, None] * dout[t].double()
    # one fp32 product (2^-24) and one bf16 rounding
    assert (gy[~held] == 7.0).all()
    assert ((gy[held].double() - want[held]).abs() <= (U + 2.0 ** -23) * want[held].abs()).all()
    dot = torch.zeros(T, k, dtype=torch.float64)
    mag = torch.zeros(T, k, dtype=torch.float64)
    dot[t, j] = (dout[t].double() * y[dst[t, j]].double()).sum(1)
    mag[t, j] = (dout[t].double() * y[dst[t, j]].double()).abs().sum(1)
    assert ((gg.double() - dot).abs() <= H * 2.0 ** -24 * mag).all()  # exact products, H additions


def test_combine_backward_reports_rows_out_of_range():
    m = _mod()
    from combine_moe_route_07_b200 import _binding
    shape = m.MoeShape(tokens=4, hidden=64, experts=4, k=2, ranks=1)
    ws = m.Workspace(shape)
    dst = torch.arange(8, dtype=torch.int32).view(4, 2)
    dst[2, 1] = 8
    y, dout = _randn(8, 64, seed=1).to(torch.bfloat16).cuda(), _randn(4, 64, seed=2).to(torch.bfloat16).cuda()
    grad_y = torch.full((8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, gg = m.moe_combine_backward(shape, dout, y, dst.cuda(), torch.ones(4, 2, device="cuda"), ws=ws,
                                   grad_y=grad_y)
    assert m.moe_get_device_error(ws) == (_binding.MOE_ERR_DEVICE_RANGE, 8)
    assert gg[2, 1] == 0 and (grad_y[5] == 7.0).all() and (gg[2, 0] != 0)
    with pytest.raises(ValueError):
        m.moe_combine_backward(shape, dout[:3], y, dst.cuda(), torch.ones(4, 2, device="cuda"), ws=ws)
    empty = m.MoeShape(tokens=0, hidden=64, experts=4, k=2, ranks=1)
    z = lambda *s, **kw: torch.empty(*s, device="cuda", **kw)  # noqa: E731
    gy, gg = m.moe_combine_backward(empty, z(0, 64, dtype=torch.bfloat16), z(0, 64, dtype=torch.bfloat16),
                                    z(0, 2, dtype=torch.int32), z(0, 2), ws=ws)
    assert gy.shape == (0, 64) and gg.shape == (0, 2)


class _Layer:
    """route -> layout -> dispatch -> swiglu product -> product -> combine + shared expert + residual."""

    def __init__(self, T, H, F, E, k, align, cap, func, seed=0):
        m = _mod()
        self.m, self.T, self.H, self.F, self.E, self.k, self.cap = m, T, H, F, E, k, cap
        self.shape = m.MoeShape(tokens=T, hidden=H, experts=E, k=k, ranks=1, align=align, capacity=cap)
        self.dense = m.MoeShape(tokens=T, hidden=H, experts=1, k=1, ranks=1)
        self.rule = m.ScoreRule(func, 4, 2, 2, 1.5)
        self.ws = m.Workspace(self.shape)
        self.wd = m.Workspace(self.dense)
        bf = lambda *s, seed, scale: _randn(*s, seed=seed, scale=scale).to(torch.bfloat16).cuda()  # noqa: E731
        self.x = bf(T, H, seed=seed + 1, scale=1.0)
        self.w1, self.w2 = bf(E, 2 * F, H, seed=seed + 2, scale=H ** -0.5), bf(E, H, F, seed=seed + 3, scale=F ** -0.5)
        self.ws1, self.ws2 = bf(1, F, H, seed=seed + 4, scale=H ** -0.5), bf(1, H, F, seed=seed + 5, scale=F ** -0.5)
        self.b1 = _randn(E, 2 * F, seed=seed + 6, scale=0.1).cuda()
        self.logits = _randn(T, E, seed=seed + 7, scale=1.5).cuda()
        self.bias = _randn(E, seed=seed + 8, scale=0.05).cuda()
        self.dout = bf(T, H, seed=seed + 9, scale=1.0)

    def step(self):
        m, sh, ws = self.m, self.shape, self.ws
        ids, gates = m.moe_route_scored(sh, self.logits, self.rule, self.bias, ws=ws)
        lay = m.moe_layout(sh, ids, ws=ws)
        rows = m.moe_dispatch(sh, self.x, lay.dst_pos, ws=ws)
        n, F, dev = sh.rows, self.F, self.x.device
        pre = torch.empty(n, 2 * F, dtype=torch.bfloat16, device=dev)
        h = m.moe_expert_matmul(sh, rows, self.w1, lay.counts, lay.expert_off, ws=ws, bias=self.b1,
                                act="swiglu", pre=pre)
        y = m.moe_expert_matmul(sh, h, self.w2, lay.counts, lay.expert_off, ws=ws)
        spre = torch.empty(self.T, F, dtype=torch.bfloat16, device=dev)
        sh1 = m.moe_expert_matmul(self.dense, self.x, self.ws1, ws=self.wd, act="gelu", pre=spre)
        shared = m.moe_expert_matmul(self.dense, sh1, self.ws2, ws=self.wd)
        out = m.moe_combine(sh, y, lay.dst_pos, gates, ws=ws, shared=shared, residual=self.x)
        # backward
        dy, dgates = m.moe_combine_backward(sh, self.dout, y, lay.dst_pos, gates, ws=ws)
        g2 = m.moe_expert_matmul_backward(sh, dy, h, self.w2, lay.counts, lay.expert_off, ws=ws)
        g1 = m.moe_expert_matmul_backward(sh, g2.grad_x, rows, self.w1, lay.counts, lay.expert_off, ws=ws,
                                          act="swiglu", pre=pre, need_bias=True)
        s2 = m.moe_expert_matmul_backward(self.dense, self.dout, sh1, self.ws2, ws=self.wd)
        s1 = m.moe_expert_matmul_backward(self.dense, s2.grad_x, self.x, self.ws1, ws=self.wd, act="gelu", pre=spre)
        ones = torch.ones(self.T, self.k, device=dev)
        dx = m.moe_combine(sh, g1.grad_x, lay.dst_pos, ones, ws=ws, shared=s1.grad_x, residual=self.dout)
        dlogits = m.moe_route_scored_backward(sh, self.logits, self.rule, ids, dgates, ws=ws)
        return {"ids": ids, "out": out, "dx": dx, "dw1": g1.grad_w, "db1": g1.grad_bias, "dw2": g2.grad_w,
                "dws1": s1.grad_w, "dws2": s2.grad_w, "dlogits": dlogits}, lay

    def exact(self, ids, dst):
        p = {n: getattr(self, n).detach().cpu().double().requires_grad_(True)
             for n in ("x", "w1", "w2", "ws1", "ws2", "b1", "logits")}
        s = torch.sigmoid(p["logits"]) if self.rule.func == "sigmoid" else torch.softmax(p["logits"], 1)
        gates = ref.gates_of(s, ids, True, self.rule.scale)
        out = p["x"] + ref.act(p["x"] @ p["ws1"][0].T, "gelu") @ p["ws2"][0].T
        add = []
        for t in range(self.T):
            for j in range(self.k):
                if dst[t, j] >= 0:
                    e = ids[t, j]
                    h = ref.act(p["x"][t] @ p["w1"][e].T + p["b1"][e], "swiglu")
                    add.append((t, gates[t, j] * (h @ p["w2"][e].T)))
        out = out.index_add(0, torch.tensor([t for t, _ in add]), torch.stack([v for _, v in add]))
        order = ["x", "w1", "b1", "w2", "ws1", "ws2", "logits"]
        grads = torch.autograd.grad(out, [p[n] for n in order], self.dout.cpu().double())
        return {"out": out.detach(), **{"d" + n: g for n, g in zip(order, grads)}}


@pytest.mark.parametrize("T,H,F,E,k,align,cap,func", [
    (70, 128, 72, 8, 3, 1, 0, "sigmoid"), (70, 128, 72, 8, 3, 16, 0, "softmax"), (60, 128, 64, 8, 3, 1, 20, "sigmoid"),
    (1, 64, 64, 8, 2, 1, 0, "sigmoid"),
])
def test_layer_and_its_gradients(T, H, F, E, k, align, cap, func):
    """Between the operators every tensor is rounded to bf16 (2^-8 each, relative): at most 8 such
    roundings lie on a path from an operand to a gradient, and a sum keeps at most their magnitude, so the
    2-norm of an error is at most 8 * 2^-8 of the 2-norm of the terms, which stays below 4 times the
    result's own for these random operands."""
    layer = _Layer(T, H, F, E, k, align, cap, func)
    got, lay = layer.step()
    layer.m.moe_check(layer.ws)
    layer.m.moe_check(layer.wd)
    ids, _, _ = ref.route(layer.logits.cpu(), k, func, True, 4, 2, 2, 1.5, layer.bias.cpu())
    assert torch.equal(got["ids"].cpu().long(), ids)
    want = layer.exact(ids, lay.dst_pos.cpu())
    for name, v in want.items():
        g = got[name].cpu().double()
        assert torch.isfinite(g).all(), name
        off = (g - v).norm() / v.norm().clamp(min=1e-12)
        assert off <= 4 * 8 * U, (name, off.item())


def test_layer_captured_and_replayed_with_new_inputs():
    layer = _Layer(200, 256, 128, 16, 4, 1, 0, "sigmoid")
    layer.step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        layer.step()
        with torch.cuda.graph(graph, stream=s):
            held, _ = layer.step()
    torch.cuda.synchronize()
    for seed in (50, 90):
        other = _Layer(200, 256, 128, 16, 4, 1, 0, "sigmoid", seed=seed)
        for n in ("x", "logits", "dout", "w1", "w2", "ws1", "ws2", "b1", "bias"):
            getattr(layer, n).copy_(getattr(other, n))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = other.step()
        torch.cuda.synchronize()
        for n, v in want.items():
            assert torch.equal(held[n], v), n
    layer.m.moe_check(layer.ws)
