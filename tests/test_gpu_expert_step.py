"""A training step of the expert layer, operator by operator: each one's output against the 64-bit formula
of the bf16 and fp32 tensors that the step itself handed it, element by element.  One operator's roundings
separate a result from its reference, so that an error in a few rows, one expert or one scale shows, where
the comparison of whole gradients (test_gpu_expert_layer.py) allows for every rounding on the way.

Tolerances as derived in test_gpu_expert_matmul.py and test_gpu_route_scored.py: u = 2^-8 for a rounding to
bf16; (K + 2) 2^-23 of the terms' magnitude for a sum of K products; 2^-18 for an activation; gates to
2^-24; a gate's gradient H 2^-24 of its terms; the logits' (2^-19 + E 2^-24) of theirs."""
import pytest
import torch

import expert_ref as ref
from test_gpu_expert_layer import _Layer
from test_gpu_expert_matmul import U, _sum_tol

pytestmark = pytest.mark.gpu


def _near(got, want, tol, what):
    got = got.cpu().double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - tol
    assert (over <= 0).all(), f"{what}: worst {over.max().item():.3g} over"


def _held(rows, segs):
    h = torch.zeros(rows, dtype=torch.bool)
    for r in segs:
        h[r] = True
    return h


def _product(x, w, segs, bias, name, got, pre, what):
    """A forward product and, with `pre`, its pre-activations, on the rows that hold a token."""
    F, K = got.shape[1], x.shape[1]
    want, z, mag = ref.matmul(x.cpu(), w.cpu(), segs, None if bias is None else bias.cpu(), name)
    zt = _sum_tol(K, mag)
    if name == "swiglu":
        gate, up = z[:, :F], z[:, F:]
        s = (gate * torch.sigmoid(gate)).abs()
        t = 1.13 * zt[:, :F] * (up.abs() + zt[:, F:]) + s * zt[:, F:] + 2.0 ** -18 * s * up.abs()
    else:
        t = 1.13 * zt + 2.0 ** -18 * (ref.act(z, name).abs() + z.abs()) * (name != "none")
    h = _held(x.shape[0], segs)
    _near(got[h.to(got.device)], want[h], (t * (1 + U) + U * want.abs())[h], what)
    if pre is not None:
        _near(pre[h.to(got.device)], z[h], (zt * (1 + U) + U * z.abs())[h], what + " pre")


def _gradients(dy, x, w, segs, g, name, pre, what):
    """A backward call: grad_pre against the formula, the products against the grad_pre that fed them."""
    F = dy.shape[1]
    dy, x, w = dy.cpu(), x.cpu(), w.cpu()
    h = _held(x.shape[0], segs)
    d = dy
    if name != "none":
        pre = pre.cpu()
        one, want = dy.double().abs(), torch.zeros(pre.shape, dtype=torch.float64)
        want[h] = ref.act_grad(pre[h].double(), dy[h].double(), name)
        slope = 4 * 2.0 ** -18 * one
        if name == "swiglu":
            zz = pre.double().abs()
            slope = torch.cat([slope * zz[:, F:], slope * (1 + zz[:, :F])], 1)
        _near(g.grad_pre.cpu()[h], want[h], (slope * (1 + U) + U * want.abs())[h], what + " grad_pre")
        if g.grad_bias is not None:
            for e, r in enumerate(segs):
                n = r.stop - r.start
                tol = slope[r].sum(0) * 1.001 + (n + 16) * 2.0 ** -24 * want[r].abs().sum(0)
                _near(g.grad_bias[e], want[r].sum(0), tol, f"{what} grad_bias of expert {e}")
        d = g.grad_pre.cpu()
    for e, r in enumerate(segs):
        n = r.stop - r.start
        de, we, xe = d[r].double(), w[e].double(), x[r].double()
        if n:
            gx, mx = de @ we, de.abs() @ we.abs()
            _near(g.grad_x[r], gx, _sum_tol(w.shape[1], mx) * (1 + U) + U * gx.abs(), f"{what} grad_x of expert {e}")
        gw, mw = de.T @ xe, de.abs().T @ xe.abs()
        _near(g.grad_w[e], gw, _sum_tol(n, mw) * (1 + U) + U * gw.abs(), f"{what} grad_w of expert {e}")


def _combined(y, dst, gates, adds, got, what):
    T, k = dst.shape
    want = sum(a.cpu().double() for a in adds)
    mag = sum(a.cpu().double().abs() for a in adds)
    for j in range(k):
        kept = dst[:, j] >= 0
        term = gates[kept, j].double()[:, None] * y.cpu()[dst[kept, j]].double()
        want[kept] += term
        mag[kept] += term.abs()
    _near(got, want, (k + 3) * 2.0 ** -24 * mag * (1 + U) + U * want.abs(), what)


@pytest.mark.parametrize("T,H,F,E,k,align,cap,func", [
    (70, 128, 72, 8, 3, 1, 0, "sigmoid"), (70, 128, 72, 8, 3, 16, 0, "softmax"),
    (60, 128, 64, 8, 3, 1, 20, "sigmoid"), (1, 64, 64, 8, 2, 1, 0, "sigmoid"),
    (900, 264, 136, 16, 4, 1, 0, "softmax"), (300, 136, 264, 24, 6, 1, 33, "softmax"),
])
def test_every_operator_of_a_step(T, H, F, E, k, align, cap, func):
    L = _Layer(T, H, F, E, k, align, cap, func)
    m, sh, ws, wd, dn = L.m, L.shape, L.ws, L.wd, L.dense
    ids, gates = m.moe_route_scored(sh, L.logits, L.rule, L.bias, ws=ws)
    lay = m.moe_layout(sh, ids, ws=ws)
    seg = (lay.counts, lay.expert_off)
    rows = m.moe_dispatch(sh, L.x, lay.dst_pos, ws=ws)
    pre = torch.empty(sh.rows, 2 * F, dtype=torch.bfloat16, device="cuda")
    h = m.moe_expert_matmul(sh, rows, L.w1, *seg, ws=ws, bias=L.b1, act="swiglu", pre=pre)
    y = m.moe_expert_matmul(sh, h, L.w2, *seg, ws=ws)
    spre = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    sh1 = m.moe_expert_matmul(dn, L.x, L.ws1, ws=wd, act="gelu", pre=spre)
    shared = m.moe_expert_matmul(dn, sh1, L.ws2, ws=wd)
    out = m.moe_combine(sh, y, lay.dst_pos, gates, ws=ws, shared=shared, residual=L.x)
    dy, dgates = m.moe_combine_backward(sh, L.dout, y, lay.dst_pos, gates, ws=ws)
    g2 = m.moe_expert_matmul_backward(sh, dy, h, L.w2, *seg, ws=ws)
    g1 = m.moe_expert_matmul_backward(sh, g2.grad_x, rows, L.w1, *seg, ws=ws, act="swiglu", pre=pre, need_bias=True)
    s2 = m.moe_expert_matmul_backward(dn, L.dout, sh1, L.ws2, ws=wd)
    s1 = m.moe_expert_matmul_backward(dn, s2.grad_x, L.x, L.ws1, ws=wd, act="gelu", pre=spre)
    ones = torch.ones(T, k, device="cuda")
    dx = m.moe_combine(sh, g1.grad_x, lay.dst_pos, ones, ws=ws, shared=s1.grad_x, residual=L.dout)
    dlogits = m.moe_route_scored_backward(sh, L.logits, L.rule, ids, dgates, ws=ws)
    m.moe_check(ws)
    m.moe_check(wd)

    want, g, _ = ref.route(L.logits.cpu(), k, func, True, 4, 2, 2, 1.5, L.bias.cpu())
    assert torch.equal(ids.cpu().long(), want)
    _near(gates, g, (2.0 ** -24 + 2.0 ** -40) * g, "gates")
    segs, dst = ref.segments(lay.counts.cpu(), lay.expert_off.cpu(), cap, E), lay.dst_pos.cpu().long()
    t, j = torch.nonzero(dst >= 0, as_tuple=True)
    at = dst[t, j]
    assert at.unique().numel() == at.numel() == int(_held(sh.rows, segs).sum())
    assert torch.equal(rows.cpu()[at], L.x.cpu()[t])
    expert_of = torch.full((sh.rows,), -1)
    for e, r in enumerate(segs):
        expert_of[r] = e
    assert torch.equal(expert_of[at], want[t, j])
    whole = [slice(0, T)]
    _product(rows, L.w1, segs, L.b1, "swiglu", h, pre, "first product")
    _product(h, L.w2, segs, None, "none", y, None, "second product")
    _product(L.x, L.ws1, whole, None, "gelu", sh1, spre, "shared first product")
    _product(sh1, L.ws2, whole, None, "none", shared, None, "shared second product")
    gc = gates.cpu()
    _combined(y, dst, gc, [shared, L.x], out, "out")

    dout, yc = L.dout.cpu().double(), y.cpu().double()
    want_dy = gc[t, j].double()[:, None] * dout[t]
    _near(dy[at.cuda()], want_dy, (U + 2.0 ** -23) * want_dy.abs(), "dy")
    dot, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    dot[t, j], mag[t, j] = (dout[t] * yc[at]).sum(1), (dout[t] * yc[at]).abs().sum(1)
    _near(dgates, dot, H * 2.0 ** -24 * mag, "dgates")
    _gradients(dy, h, L.w2, segs, g2, "none", None, "second product")
    _gradients(g2.grad_x, rows, L.w1, segs, g1, "swiglu", pre, "first product")
    _gradients(L.dout, sh1, L.ws2, whole, s2, "none", None, "shared second product")
    _gradients(s2.grad_x, L.x, L.ws1, whole, s1, "gelu", spre, "shared first product")
    _combined(g1.grad_x, dst, torch.ones(T, k), [s1.grad_x, L.dout], dx, "dx")

    z = L.logits.cpu().double().requires_grad_(True)
    s = torch.sigmoid(z) if func == "sigmoid" else torch.softmax(z, 1)
    up = dgates.cpu().double()
    dl = torch.autograd.grad(ref.gates_of(s, want, True, 1.5), z, up)[0]
    part = torch.zeros(T, E, dtype=torch.float64).scatter_(1, want, g * up.abs())
    share = torch.zeros(T, E, dtype=torch.float64).scatter_(1, want, torch.gather(s.detach(), 1, want))
    total = (g * up.abs()).sum(1, keepdim=True)
    part = part + share / share.sum(1, keepdim=True) * total
    _near(dlogits, dl, (2.0 ** -19 + E * 2.0 ** -24) * part + 2.0 ** -42 * total, "dlogits")
