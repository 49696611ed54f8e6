"""Host-side checks of the scored route, the experts' products and the gradients: every refusal comes
before any CUDA call, so no GPU is needed (the pointers are never followed)."""
import ctypes

import pytest

from combine_moe_route_07_b200 import _binding

FAKE = 0x10000
BIG = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from combine_moe_route_07_b200 import build
    build.build()
    return _binding.lib()


def _shape(**kw):
    base = dict(tokens=64, hidden=256, experts=16, k=4, ranks=1, capacity=0, align=1, flags=1)
    base.update(kw)
    return _binding.MoeShapeC(**base)


def _rule(**kw):
    base = dict(func=1, groups=4, top_groups=2, group_top=2, scale=1.0)
    base.update(kw)
    return _binding.MoeScoreC(**base)


def _route(lib, s=None, r=None, logits=FAKE, bias=None, ids=FAKE, gates=FAKE, ws=FAKE, nbytes=BIG, null_rule=False):
    s = s or _shape()
    return lib.moe_route_scored(ctypes.byref(s), logits, bias, None if null_rule else ctypes.byref(r or _rule()), ids,
                                gates, ws, nbytes, None)


def _route_back(lib, s=None, r=None, logits=FAKE, ids=FAKE, gg=FAKE, out=FAKE, ws=FAKE, nbytes=BIG):
    s = s or _shape()
    return lib.moe_route_scored_backward(ctypes.byref(s), logits, ctypes.byref(r or _rule()), ids, gg, out, ws, nbytes,
                                         None)


@pytest.mark.parametrize("bad", [
    dict(func=2), dict(func=-1), dict(groups=0), dict(groups=3), dict(groups=128), dict(top_groups=0),
    dict(top_groups=5), dict(group_top=0), dict(group_top=3), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(groups=16, top_groups=8, group_top=2),
    dict(groups=16, top_groups=3, group_top=1),  # 3 experts for k = 4
])
def test_bad_rules_are_refused(lib, bad):
    assert _route(lib, r=_rule(**bad)) == 1
    assert _route_back(lib, r=_rule(**bad)) == 1


def test_rule_with_more_than_64_groups_is_refused(lib):
    s = _shape(experts=256)
    assert _route(lib, s=s, r=_rule(groups=128, top_groups=64, group_top=2)) == 1


def test_scored_route_pointers_and_workspace(lib):
    assert _route(lib, null_rule=True) == 1
    for kw in (dict(logits=None), dict(ids=None), dict(gates=None), dict(logits=FAKE + 2), dict(bias=FAKE + 1),
               dict(ids=FAKE + 2), dict(gates=FAKE + 3)):
        assert _route(lib, **kw) == 1, kw
    for kw in (dict(logits=None), dict(ids=None), dict(gg=None), dict(out=None), dict(out=FAKE + 2)):
        assert _route_back(lib, **kw) == 1, kw
    for f in (_route, _route_back):
        assert f(lib, ws=None) == 3
        assert f(lib, ws=FAKE + 8) == 3
        assert f(lib, nbytes=64) == 3
        assert f(lib, s=_shape(k=17)) == 1
        assert f(lib, s=_shape(tokens=0)) == 0  # nothing to do, nothing launched


def _matmul(lib, s=None, k=256, f=128, act=0, x=FAKE, w=FAKE, bias=None, counts=FAKE, off=FAKE, res=None, out=FAKE,
            pre=None, ws=FAKE, nbytes=BIG):
    s = s or _shape()
    return lib.moe_expert_matmul(ctypes.byref(s), k, f, act, x, w, bias, counts, off, res, out, pre, ws, nbytes, None)


def _matmul_back(lib, s=None, k=256, f=128, act=0, dy=FAKE, x=FAKE, w=FAKE, pre=None, counts=FAKE, off=FAKE, gp=None,
                 gx=FAKE, gw=FAKE, gb=None, scratch=None, sbytes=0, ws=FAKE, nbytes=BIG):
    s = s or _shape()
    return lib.moe_expert_matmul_backward(ctypes.byref(s), k, f, act, dy, x, w, pre, counts, off, gp, gx, gw, gb,
                                          scratch, sbytes, ws, nbytes, None)


@pytest.mark.parametrize("call", [_matmul, _matmul_back])
@pytest.mark.parametrize("bad", [
    dict(k=0), dict(k=12), dict(k=65544), dict(f=0), dict(f=4), dict(f=20), dict(f=65544), dict(act=-1), dict(act=5),
    dict(counts=None), dict(off=None), dict(counts=None, off=None), dict(counts=FAKE + 2), dict(off=FAKE + 1),
    dict(x=FAKE + 8), dict(w=FAKE + 8), dict(x=None), dict(w=None),
    dict(s=_shape(flags=5)), dict(s=_shape(k=17)), dict(s=_shape(hidden=12)),
])
def test_bad_products_are_refused(lib, call, bad):
    assert call(lib, **bad) == 1


def test_dense_products_need_one_dropless_expert(lib):
    dense = dict(counts=None, off=None)
    for s in (_shape(experts=2, k=1), _shape(experts=1, k=1, capacity=8), _shape(experts=1, k=1, align=8)):
        assert _matmul(lib, s=s, **dense) == 1
        assert _matmul_back(lib, s=s, **dense) == 1
    empty = _shape(experts=1, k=1, tokens=0)
    assert _matmul(lib, s=empty, **dense) == 0


def test_product_pointers_and_workspace(lib):
    for kw in (dict(out=None), dict(out=FAKE + 8), dict(pre=FAKE + 8), dict(res=FAKE + 8), dict(bias=FAKE + 2)):
        assert _matmul(lib, **kw) == 1, kw
    for kw in (dict(dy=None), dict(act=2), dict(act=2, pre=FAKE), dict(act=2, gp=FAKE), dict(gx=FAKE + 8),
               dict(gw=FAKE + 8), dict(gb=FAKE + 2, scratch=FAKE, sbytes=BIG), dict(gp=FAKE + 8)):
        assert _matmul_back(lib, **kw) == 1, kw
    for f in (_matmul, _matmul_back):
        assert f(lib, ws=None) == 3
        assert f(lib, nbytes=64) == 3
    # the bias gradient needs its scratch
    need = lib.moe_expert_matmul_backward_scratch_bytes(ctypes.byref(_shape()), 128, 0)
    assert _matmul_back(lib, gb=FAKE) == 3
    assert _matmul_back(lib, gb=FAKE, scratch=FAKE, sbytes=need - 1) == 3


def test_too_many_tiles_are_unsupported(lib):
    # 2^29 assignments of 65536 features: more tiles than the kernels can number
    s = _shape(tokens=1 << 27, experts=4, k=4, hidden=8)
    assert _matmul(lib, s=s, f=65536) == 2
    assert _matmul_back(lib, s=s, f=65536) == 2


def test_scratch_bytes(lib):
    f = lambda s, n, act: lib.moe_expert_matmul_backward_scratch_bytes(ctypes.byref(s), n, act)  # noqa: E731
    # the experts' first tiles (17 words, in 16-byte pieces), and a row of sums for at most
    # T*k/64 + min(E, T*k) tiles
    assert f(_shape(), 128, 0) == 80 + (256 // 64 + 16) * 128 * 4
    assert f(_shape(), 128, 4) == 80 + (256 // 64 + 16) * 256 * 4
    assert f(_shape(tokens=1, k=2), 128, 0) == 80 + 2 * 128 * 4
    for bad in (f(_shape(), 12, 0), f(_shape(), 128, 9), f(_shape(flags=5), 128, 0), f(_shape(k=99), 128, 0)):
        assert bad == 0


def test_combine_backward_is_checked(lib):
    def call(s=None, do=FAKE, y=FAKE, dst=FAKE, g=FAKE, gy=FAKE, gg=FAKE, ws=FAKE, nbytes=BIG):
        s = s or _shape()
        return lib.moe_combine_backward(ctypes.byref(s), do, y, dst, g, gy, gg, ws, nbytes, None)

    for kw in (dict(do=None), dict(y=None), dict(dst=None), dict(g=None), dict(gy=None), dict(gg=None),
               dict(do=FAKE + 8), dict(y=FAKE + 8), dict(gy=FAKE + 8), dict(dst=FAKE + 2), dict(g=FAKE + 1),
               dict(gg=FAKE + 2), dict(s=_shape(hidden=12))):
        assert call(**kw) == 1, kw
    assert call(ws=None) == 3 and call(nbytes=16) == 3
    assert call(s=_shape(tokens=0)) == 0


def test_python_names():
    import combine_moe_route_07_b200 as m
    for name in ("ScoreRule", "ExpertGrads", "moe_route_scored", "moe_route_scored_backward", "moe_expert_matmul",
                 "moe_expert_matmul_backward", "moe_combine_backward"):
        assert name in m.__all__ and hasattr(m, name)
    with pytest.raises(ValueError):
        m.ScoreRule("tanh").c()
    assert m.ScoreRule("sigmoid", 8, 4, 2, 2.5).c().scale == 2.5
