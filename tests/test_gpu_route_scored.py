"""moe_route_scored and its gradient against the 64-bit definition: scores, groups, ties, masked and
infinite logits, saturated scores, NaN rows, every size class; the gradient against the formulas and
against differences.

Ids are compared exactly: keys are those of binary64 arithmetic.  Gates: with renormalisation, or with
sigmoid scores, they are quotients of binary64 scores rounded once to fp32 (2^-24, and 2^-40 for the
binary64 steps); the full softmax's sum of up to 1024 exponentials is held to 1e-6, the tolerance of the
library's other gates.
"""
import pytest
import torch

import expert_ref as ref

pytestmark = pytest.mark.gpu


def _mod():
    import combine_moe_route_07_b200 as m
    return m


def _gate_tol(func, renorm):
    return 1e-6 if func == "softmax" and not renorm else 2.0 ** -24 + 2.0 ** -40


def _run(logits, k, func, renorm, groups=1, top=1, gt=1, scale=1.0, bias=None, check=True):
    m = _mod()
    T, E = logits.shape
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1, renorm=renorm)
    ws = m.Workspace(shape)
    rule = m.ScoreRule(func, groups, top, gt, scale)
    ids, gates = m.moe_route_scored(shape, logits.cuda(), rule, None if bias is None else bias.cuda(), ws=ws)
    if check:
        m.moe_check(ws)
    return ids.cpu(), gates.cpu(), ws


def _compare(logits, k, func, renorm, groups=1, top=1, gt=1, scale=1.0, bias=None):
    ids, gates, _ = _run(logits, k, func, renorm, groups, top, gt, scale, bias)
    want, g, _ = ref.route(logits, k, func, renorm, groups, top, gt, scale, bias)
    assert torch.equal(ids.long(), want)
    tol = _gate_tol(func, renorm) * g.abs() + 2.0 ** -140  # gates below fp32's normal range
    assert ((gates.double() - g).abs() <= tol).all()


def _randn(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top,gt", [
    (300, 8, 2, 1, 1, 1), (257, 64, 6, 8, 3, 2), (500, 256, 8, 8, 4, 2), (333, 512, 10, 8, 4, 2),
    (129, 256, 8, 16, 3, 1), (65, 1024, 32, 1, 1, 1), (64, 1024, 16, 64, 5, 2), (77, 96, 5, 6, 2, 2),
    (90, 100, 7, 4, 3, 1), (50, 33, 4, 1, 1, 1), (40, 160, 8, 10, 9, 2), (31, 5, 5, 5, 5, 1), (1, 256, 8, 8, 4, 2),
    (12, 1, 1, 1, 1, 1), (200, 384, 8, 8, 4, 2), (200, 128, 8, 64, 8, 2), (100, 320, 6, 2, 1, 2),
])
def test_random(func, renorm, with_bias, T, E, k, groups, top, gt):
    bias = _randn(E, seed=9, scale=0.05) if with_bias else None
    _compare(_randn(T, E, seed=T + E, scale=1.5), k, func, renorm, groups, top, gt, 2.5, bias)


@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,gt", [(1, 1, 1), (8, 3, 2), (8, 4, 1)])
def test_ties_take_the_lower_index(func, groups, top, gt):
    E, k = 64, 6
    g = torch.Generator().manual_seed(4)
    rows = [torch.zeros(E), torch.ones(E) * -3.0]
    rows += [torch.randint(0, n, (E,), generator=g).float() * 0.5 for n in (2, 3, 5, 9) for _ in range(40)]
    rows.append(torch.tensor([0.0, -0.0] * (E // 2)))
    _compare(torch.stack(rows), k, func, True, groups, top, gt)
    # bias that makes different logits nearly, not exactly, equal keys
    logits = _randn(200, E, seed=5)
    s = ref.scores(logits, func)
    _compare(logits, k, func, False, groups, top, gt, bias=(0.5 - s[0]).float())


def test_neighbouring_keys_are_ordered_exactly():
    """Logits one fp32 step apart around a common value: fp32 scores would tie."""
    base = torch.tensor(0.75).view(torch.int32)
    g = torch.Generator().manual_seed(6)
    rows = [(base + torch.randperm(256, generator=g).int()).view(torch.float32) for _ in range(64)]
    for func in ("softmax", "sigmoid"):
        for groups, top, gt in ((1, 1, 1), (8, 4, 2)):
            _compare(torch.stack(rows), 8, func, True, groups, top, gt)
            _compare(torch.stack(rows), 8, func, True, groups, top, gt, bias=torch.full((256,), 0.125))


def test_masked_and_saturated_logits():
    E = 128
    logits = _randn(300, E, seed=7, scale=2.0)
    for t in range(300):  # all but t % 12 + 1 experts masked
        logits[t, torch.randperm(E, generator=torch.Generator().manual_seed(t))[t % 12 + 1:]] = -float("inf")
    for func in ("softmax", "sigmoid"):
        _compare(logits, 6, func, True, 8, 4, 2)
        _compare(logits, 6, func, False)
    lowest = torch.where(torch.isinf(logits), torch.finfo(torch.float32).min, logits)
    for func in ("softmax", "sigmoid"):
        _compare(lowest, 6, func, True, 8, 4, 2)
    # sigmoid of large logits is 1 in fp32 long before it is in binary64
    _compare(_randn(100, E, seed=8, scale=30.0), 6, "sigmoid", True, 8, 4, 2)
    _compare(_randn(100, E, seed=8, scale=300.0), 6, "softmax", True, 8, 4, 2)
    _compare(_randn(100, E, seed=8, scale=1e-6), 6, "sigmoid", True, 8, 4, 2)
    # nothing left: every sigmoid score is zero, gates are zero
    ids, gates, _ = _run(torch.full((3, E), -float("inf")), 6, "sigmoid", True)
    assert torch.equal(ids, torch.arange(6, dtype=torch.int32).expand(3, 6)) and (gates == 0).all()


def test_bias_of_minus_infinity_excludes():
    E = 64
    logits, bias = _randn(100, E, seed=3), torch.zeros(E)
    bias[torch.randperm(E, generator=torch.Generator().manual_seed(1))[:50]] = -float("inf")
    for func in ("softmax", "sigmoid"):
        _compare(logits, 8, func, True, bias=bias)
        _compare(logits, 16, func, True, bias=bias)  # 14 experts left, then the lowest ids
        _compare(logits, 8, func, True, 8, 2, 2, bias=bias)


def test_nan_rows_are_reported_and_stay_valid():
    m = _mod()
    from combine_moe_route_07_b200 import _binding
    for func, value in (("sigmoid", float("nan")), ("softmax", float("nan")), ("softmax", float("inf"))):
        for E in (64, 256, 512):
            logits = _randn(40, E, seed=2)
            logits[17, E - 3] = value
            ids, gates, ws = _run(logits, 4, func, True, check=False)
            assert m.moe_get_device_error(ws) == (_binding.MOE_ERR_DEVICE_NAN, 17)
            assert ids[17].tolist() == [0, 1, 2, 3] and (gates[17] == 0).all()
            keep = [t for t in range(40) if t != 17]
            want, g, _ = ref.route(logits[keep], 4, func, True)
            assert torch.equal(ids[keep].long(), want)
    ids, gates, ws = _run(torch.full((2, 64), -float("inf")), 4, "softmax", True, check=False)
    assert m.moe_get_device_error(ws)[0] == _binding.MOE_ERR_DEVICE_NAN
    ids, gates, ws = _run(_randn(2, 64), 4, "sigmoid", True, check=False,
                          bias=torch.full((64,), float("inf")))
    assert m.moe_get_device_error(ws)[0] == _binding.MOE_ERR_DEVICE_NAN


def test_skewed_popularity_and_large_batch():
    logits = _randn(20000, 512, seed=12) - 2.0 * torch.log(torch.arange(1, 513).float())
    _compare(logits, 10, "sigmoid", True, 8, 4, 2, 2.5, _randn(512, seed=13, scale=0.05))
    _compare(logits, 10, "softmax", True)
    _compare(logits, 10, "softmax", False, bias=_randn(512, seed=13, scale=0.01))


@pytest.mark.parametrize("func,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                         ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 2), (300, 64, 6), (257, 256, 8), (129, 515, 10),
                                   (50, 1024, 32)])
def test_gradient(func, renorm, T, E, k):
    """fp32 steps: scores are off by at most 2^-20 relative, sums of k (or E) terms by (k or E) 2^-24, so
    each part by 2^-19 + E 2^-24 of the magnitude of the terms it is a difference of.  The oracle goes
    through the full softmax, whose two contributions to an expert outside the choice cancel only to
    their 64-bit rounding: at most E + k steps of 2^-53 of the sum of the terms, below 2^-42 of it."""
    m = _mod()
    logits, up = _randn(T, E, seed=1, scale=1.5), _randn(T, k, seed=2)
    ids, _, _ = ref.route(logits, k, func, renorm)
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1, renorm=renorm)
    ws = m.Workspace(shape)
    got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule(func, scale=2.5),
                                      ids.int().cuda(), up.cuda(), ws=ws).cpu()
    m.moe_check(ws)
    z = logits.double().requires_grad_(True)
    s = torch.sigmoid(z) if func == "sigmoid" else torch.softmax(z, 1)
    gates = ref.gates_of(s, ids, renorm, 2.5)
    want = torch.autograd.grad(gates, z, up.double())[0]
    g = gates.detach().abs()
    mag = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, g * up.double().abs())
    total = (g * up.double().abs()).sum(1, keepdim=True)
    share = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ids, torch.gather(s.detach(), 1, ids))
    if renorm:
        share = share / share.sum(1, keepdim=True)
    elif func == "softmax":
        share = s.detach()
    mag = mag + share * total
    assert ((got.double() - want).abs() <= (2.0 ** -19 + E * 2.0 ** -24) * mag + 2.0 ** -42 * total
            + 2.0 ** -140).all()
    if renorm or func == "sigmoid":
        off = torch.ones(T, E, dtype=torch.bool).scatter_(1, ids, False)
        assert (got[off] == 0).all()


def test_gradient_agrees_with_differences():
    m = _mod()
    T, E, k = 4, 12, 3
    logits, up = _randn(T, E, seed=1), _randn(T, k, seed=2)
    for func in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _, _ = ref.route(logits, k, func, renorm)
            shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1, renorm=renorm)
            got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule(func), ids.int().cuda(),
                                              up.cuda(), ws=m.Workspace(shape)).cpu()
            for e in range(E):
                h = torch.zeros(E, dtype=torch.float64)
                h[e] = 1e-5
                f = [(ref.gates_of(ref.scores(logits.double() + q * h, func), ids, renorm, 1.0) * up).sum(1)
                     for q in (1, -1)]
                assert ((got[:, e].double() - (f[0] - f[1]) / 2e-5).abs() <= 1e-5).all()


def test_gradient_edges():
    m = _mod()
    from combine_moe_route_07_b200 import _binding
    T, E, k = 5, 40, 4
    logits, up = _randn(T, E, seed=1), _randn(T, k, seed=2)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    ids[0] = torch.tensor([7, 3, 7, 7])  # one expert in three slots
    ids[1] = torch.tensor([E, 2, 9, 11])  # outside
    ids[2] = torch.tensor([5, -1, 6, 8])
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1, renorm=False)
    ws = m.Workspace(shape)
    got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule("sigmoid"), ids.cuda(), up.cuda(),
                                      ws=ws).cpu()
    assert m.moe_get_device_error(ws)[0] == _binding.MOE_ERR_DEVICE_RANGE
    ok = (ids >= 0) & (ids < E)
    s = torch.sigmoid(logits.double())
    at = ids.clamp(0, E - 1).long()
    part = torch.where(ok, up.double() * torch.gather(s * (1 - s), 1, at), 0.0)
    want = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, at, part)
    assert ((got.double() - want).abs() <= 2.0 ** -19 * up.double().abs().sum(1, keepdim=True)).all()
    # saturated and masked: finite gradients, zero where the score is
    logits = torch.full((2, E), -float("inf"))
    logits[1] = 200.0
    ids = torch.arange(k, dtype=torch.int32).expand(2, k).contiguous()
    for renorm in (False, True):
        shape = m.MoeShape(tokens=2, hidden=8, experts=E, k=k, ranks=1, renorm=renorm)
        got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule("sigmoid"), ids.cuda(),
                                          up[:2].cuda(), ws=m.Workspace(shape)).cpu()
        assert (got.abs() <= 2.0 ** -100).all()


@pytest.mark.parametrize("E,groups,k", [(64, 2, 6), (128, 4, 8), (256, 8, 8), (512, 8, 10), (512, 16, 9),
                                        (1024, 32, 8), (512, 2, 32), (160, 5, 6), (96, 8, 5), (80, 16, 4)])
@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
def test_groups_closer_than_fp32_are_decided_exactly(func, E, groups, k):
    """Every group holds the same values in another order, some moved by one fp32 step: which groups are
    kept is a matter of the last bits, or of the lower index."""
    g = torch.Generator().manual_seed(E + groups)
    T, G = 64, E // groups
    base = torch.randn(T, 1, G, generator=g).expand(T, groups, G)
    order = torch.rand(T, groups, G, generator=g).argsort(2)
    logits = torch.gather(base, 2, order).reshape(T, E)
    moved = torch.rand(T, E, generator=g) < 0.2
    logits = torch.where(moved, torch.nextafter(logits, torch.full_like(logits, 9.0)), logits)
    top = max(1, groups // 2)
    for gt in (1, 2):
        if top * G >= k:
            for bias in (None, torch.full((E,), 0.125)):
                _compare(logits, k, func, True, groups, top, gt, 1.0, bias)


@pytest.mark.parametrize("E,groups", [(64, 8), (128, 4), (256, 8), (512, 8), (512, 32), (160, 5)])
def test_nan_in_any_group_is_reported(E, groups):
    m = _mod()
    from combine_moe_route_07_b200 import _binding
    logits = _randn(12, E, seed=groups)
    for e in range(0, E, max(1, E // 13)):
        bad = logits.clone()
        bad[5] -= 4.0 * (torch.arange(E) // (E // groups) == e * groups // E)  # its group is not among the best
        bad[5, e] = float("nan")
        for func in ("sigmoid", "softmax"):
            ids, gates, ws = _run(bad, 4, func, True, groups, groups // 2, 2, check=False)
            assert m.moe_get_device_error(ws) == (_binding.MOE_ERR_DEVICE_NAN, 5)
            assert ids[5].tolist() == [0, 1, 2, 3] and (gates[5] == 0).all()
            keep = [t for t in range(12) if t != 5]
            want, _, _ = ref.route(logits[keep], 4, func, True, groups, groups // 2, 2)
            assert torch.equal(ids[keep].long(), want)


def test_gradient_of_scores_below_fp32():
    """Sigmoid scores whose chosen sum is near or below fp32's smallest number: the gates are quotients
    of them all the same, and so are the gradients."""
    m = _mod()
    T, E, k = 96, 64, 5
    top = torch.linspace(-60.0, -600.0, T)[:, None]
    logits = top + _randn(T, E, seed=4)
    up = _randn(T, k, seed=5)
    logits[7] = -800.0  # scores that binary64 loses too: gates and gradients of zero
    ids, gates, _ = _run(logits, k, "sigmoid", True)
    _compare(logits, k, "sigmoid", True)
    assert (gates[7] == 0).all()
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1, renorm=True)
    got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule("sigmoid"), ids.int().cuda(),
                                      up.cuda(), ws=m.Workspace(shape)).cpu().double()
    at = ids.cpu().long()
    s = ref.scores(torch.gather(logits, 1, at), "sigmoid")
    total = s.sum(1, keepdim=True)
    q = torch.where(total > 0, s / total, torch.zeros_like(s))
    part = q * (up.double() - (q * up.double()).sum(1, keepdim=True)) * (1.0 - s)
    want = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, at, part)
    # quotients within 2^-21 (exp and the division in fp32), their weighted sum of k parts likewise
    assert ((got - want).abs() <= 2.0 ** -19 * up.double().abs().sum(1, keepdim=True)).all()
    assert (got[7] == 0).all() and (got[T - 1] != 0).any()


def test_a_bias_that_chooses_masked_experts():
    """Softmax over masked logits: a bias can choose experts of score zero alone."""
    m = _mod()
    T, E, k = 6, 48, 4
    for W in (k, 20):  # both sizes of a token's lane group
        logits = _randn(T, E, seed=1)
        logits[:, :W] = -float("inf")
        bias = torch.zeros(E)
        bias[:W] = 3.0 - 0.01 * torch.arange(W)
        ids, gates, _ = _run(logits, W, "softmax", True, bias=bias)
        assert (gates == 0).all() and torch.equal(ids.cpu().long(), torch.arange(W).expand(T, W))
        shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=W, ranks=1, renorm=True)
        got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule("softmax"), ids.int().cuda(),
                                          _randn(T, W, seed=2).cuda(), ws=m.Workspace(shape))
        assert (got == 0).all()


def test_unaligned_rows_and_other_stream():
    """Logits and outputs that start 4 bytes behind a 16-byte boundary, on a stream of their own."""
    m = _mod()
    T, E, k = 70, 256, 8
    base = _randn(T * E + 1, seed=1).cuda()
    logits = base[1:].view(T, E)
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1)
    ws = m.Workspace(shape)
    rule = m.ScoreRule("sigmoid", 8, 4, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids, gates = m.moe_route_scored(shape, logits, rule, ws=ws)
        grad = torch.full((T * E + 1,), 9.0, device="cuda")
        m.moe_route_scored_backward(shape, logits, rule, ids, gates, ws=ws, grad_logits=grad[1:].view(T, E))
    s.synchronize()
    want, _, _ = ref.route(logits.cpu(), k, "sigmoid", True, 8, 4, 2)
    assert torch.equal(ids.cpu().long(), want)
    whole = m.moe_route_scored_backward(shape, logits.clone(), rule, ids, gates, ws=ws)
    assert torch.equal(grad[1:].view(T, E), whole) and grad[0] == 9.0


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens' rows are where they belong."""
    m = _mod()
    T, E, k = (1 << 21) + 37, 1024, 4
    logits = torch.randn(1 << 14, E, device="cuda").repeat(T // (1 << 14) + 1, 1)[:T].contiguous()
    logits[-64:] = _randn(64, E, seed=5).cuda()
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1)
    ws = m.Workspace(shape)
    rule = m.ScoreRule("sigmoid", 8, 4, 2)
    ids, gates = m.moe_route_scored(shape, logits, rule, ws=ws)
    m.moe_check(ws)
    want, g, _ = ref.route(logits[-64:].cpu(), k, "sigmoid", True, 8, 4, 2)
    assert torch.equal(ids[-64:].cpu().long(), want)
    assert ((gates[-64:].cpu().double() - g).abs() <= _gate_tol("sigmoid", True) * g).all()
    grad = m.moe_route_scored_backward(shape, logits, rule, ids, gates, ws=ws)
    m.moe_check(ws)
    del logits
    assert torch.isfinite(grad[-64:]).all()
    off = torch.ones(64, E, dtype=torch.bool, device="cuda").scatter_(1, ids[-64:].long(), False)
    assert (grad[-64:][off] == 0).all() and (grad[-64:][~off] != 0).any()
    assert int((grad[: 1 << 14] != 0).sum()) <= (1 << 14) * k


def test_no_tokens_and_wrong_arguments():
    m = _mod()
    shape = m.MoeShape(tokens=0, hidden=8, experts=8, k=2, ranks=1)
    ws = m.Workspace(shape)
    ids, gates = m.moe_route_scored(shape, torch.empty(0, 8, device="cuda"), m.ScoreRule(), ws=ws)
    assert ids.shape == (0, 2) and gates.shape == (0, 2)
    shape = m.MoeShape(tokens=4, hidden=8, experts=8, k=2, ranks=1)
    logits = torch.zeros(4, 8, device="cuda")
    for rule in (m.ScoreRule(groups=3), m.ScoreRule(groups=0), m.ScoreRule(groups=4, top_groups=5),
                 m.ScoreRule(groups=8, top_groups=1), m.ScoreRule(group_top=3), m.ScoreRule(group_top=0),
                 m.ScoreRule(groups=8, top_groups=4, group_top=2), m.ScoreRule(scale=0.0),
                 m.ScoreRule(scale=float("nan"))):
        with pytest.raises(m.MoeError):
            m.moe_route_scored(shape, logits, rule, ws=ws)
    with pytest.raises(ValueError):
        m.moe_route_scored(shape, logits, m.ScoreRule("relu"), ws=ws)
    with pytest.raises(ValueError):
        m.moe_route_scored(shape, logits.cpu(), m.ScoreRule(), ws=ws)
    with pytest.raises(ValueError):
        m.moe_route_scored(shape, logits.t().contiguous().t(), m.ScoreRule(), ws=ws)


def _masked_choice(T, E, W, value, seed):
    """Logits whose first W experts are far below the others in all but every third token, and a bias that
    chooses just those W."""
    logits = _randn(T, E, seed=seed)
    low = torch.arange(T) % 3 != 2
    logits[low, :W] = value if abs(value) > 1e6 else logits[low, :W] + value
    bias = torch.zeros(E)
    bias[:W] = 3.0 - 0.01 * torch.arange(W)
    return logits, bias


@pytest.mark.parametrize("value", [-1e9, torch.finfo(torch.float32).min, -800.0, -600.0, -90.0])
@pytest.mark.parametrize("E,W", [(48, 4), (51, 5), (256, 16), (64, 20), (1024, 32)])
@pytest.mark.parametrize("shift", [0.0, 300.0])
def test_gradient_where_the_chosen_scores_vanish(value, E, W, shift):
    """Experts masked with a finite value, chosen by a bias: where the scores are zero in binary64 the gates
    are zero whatever the logits, and so are the gradients.  Scores that binary64 still holds (600 below the
    largest logit) have gates and gradients like any others.  Quotients: expf of a difference of logits below
    8 (2^-21) and fp32 sums of up to 32 terms (2^-19), as in the other gradient tests."""
    m = _mod()
    T = 41
    logits, bias = _masked_choice(T, E, W, value, E + W)
    logits = logits + shift
    up = _randn(T, W, seed=2)
    want, g, _ = ref.route(logits, W, "softmax", True, bias=bias)
    ids, gates, _ = _run(logits, W, "softmax", True, bias=bias)
    assert torch.equal(ids.long(), want)
    gone = (g == 0).all(1)
    assert int(gone.sum()) == (T - T // 3 if value <= -800.0 else 0)
    assert (gates[gone] == 0).all()
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=W, ranks=1, renorm=True)
    got = m.moe_route_scored_backward(shape, logits.cuda(), m.ScoreRule("softmax"), ids.cuda(), up.cuda(),
                                      ws=m.Workspace(shape)).cpu().double()
    part = g * (up.double() - (g * up.double()).sum(1, keepdim=True))
    whole = torch.zeros(T, E, dtype=torch.float64).scatter_(1, want, part)
    assert ((got - whole).abs() <= 2.0 ** -18 * up.double().abs().sum(1, keepdim=True)).all()
    assert (got[gone] == 0).all()


@pytest.mark.parametrize("E,W", [(48, 4), (300, 16), (1000, 24)])
def test_gates_of_scores_at_the_end_of_binary64(E, W):
    """Chosen scores that are binary64's last few subnormals, or the first that it loses: the gates are
    quotients of those numbers, as everywhere."""
    T = 200
    logits = _randn(T, E, seed=E, scale=0.3)
    logits[:, :W] = torch.linspace(-725.0, -748.0, T)[:, None] + _randn(T, W, seed=1, scale=0.3)
    bias = torch.zeros(E)
    bias[:W] = 3.0 - 0.01 * torch.arange(W)
    want, g, _ = ref.route(logits, W, "softmax", True, bias=bias)
    assert (g == 0).all(1).any() and not (g == 0).all(1).all()
    _compare(logits, W, "softmax", True, bias=bias)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(40, 4), (37, 20), (1024, 32)])
def test_gradient_of_a_row_whose_mask_leaves_nothing(renorm, E, k):
    """Every logit -inf: the route reports the token and gives it gates of zero; it has no gradient, and the
    tokens beside it have theirs."""
    m = _mod()
    T = 9
    logits, up = _randn(T, E, seed=3), _randn(T, k, seed=4)
    logits[[0, 4]] = -float("inf")
    ids = torch.arange(k, dtype=torch.int32).expand(T, k).contiguous()
    shape = m.MoeShape(tokens=T, hidden=8, experts=E, k=k, ranks=1, renorm=renorm)
    call = lambda l: m.moe_route_scored_backward(  # noqa: E731
        shape, l.cuda(), m.ScoreRule("softmax"), ids.cuda(), up.cuda(), ws=m.Workspace(shape)).cpu()
    got = call(logits)
    assert (got[[0, 4]] == 0).all()
    keep = [t for t in range(T) if t not in (0, 4)]
    other = logits.clone()
    other[[0, 4]] = 1.0
    assert torch.equal(got[keep], call(other)[keep]) and (got[keep] != 0).any()


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E", [64, 256, 512, 1024])
def test_softmax_gates_over_nearly_equal_logits(E, with_bias):
    """Gates without renormalisation where every rounding of the sum's terms goes one way: one expert
    ahead of E - 1 equal ones."""
    T = 4096
    ahead = torch.linspace(0.0, 12.0, T)
    logits = torch.zeros(T, E)
    logits[:, 5] = ahead
    base = _randn(T, 1, seed=E, scale=3.0)
    bias = 0.01 * _randn(E, seed=1) if with_bias else None
    _compare(logits + base, 4, "softmax", False, bias=bias)
    _compare(-logits.flip(1) - base, 4, "softmax", False, bias=bias)


@pytest.mark.parametrize("shift", [0.0, -77.7, 313.1, -5001.3, 32760.9, -40000.3, 3e6])
@pytest.mark.parametrize("renorm", [False, True])
def test_softmax_of_shifted_logits(shift, renorm):
    """Rows whose largest logit is far from zero, and a bias that brings their keys within 1e-6 of each
    other: the choice and the gates are the 64-bit ones of the shifted values."""
    for E, groups, top, gt in ((64, 1, 1, 1), (256, 8, 4, 2), (512, 1, 1, 1), (100, 4, 2, 1)):
        T = 300
        logits = _randn(T, E, seed=E, scale=1.5) + shift
        _compare(logits, 6, "softmax", renorm, groups, top, gt)
        s = ref.scores(logits[:1], "softmax")[0]
        near = (s + 1e-6 * _randn(E, seed=3).double())
        row = logits[:1].expand(T, E).clone()
        row[:, 1::2] = row[:, 1::2] + 1e-3 * _randn(T, E // 2, seed=4)  # the sums differ, most keys stay near
        _compare(row, 6, "softmax", renorm, groups, top, gt, bias=(0.5 - near).float())
