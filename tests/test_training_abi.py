"""Host checks of the training entry points (no GPU): bad arguments are refused before the device is touched,
and CPU tensors before the library is called."""
import ctypes

import pytest

from ternary_weight_linear_fwd_b200 import build as blbuild

NULL, SHAPE, ALIGN, PATTERN, FLAGS = 1, 2, 3, 4, 8
P = 1 << 20  # an aligned address that nothing reads: every call below is refused on the host


@pytest.fixture(scope="module")
def L():
    blbuild.build()
    import ternary_weight_linear_fwd_b200 as bl
    return bl.lib()


def _weights(**kw):
    import ternary_weight_linear_fwd_b200 as bl
    d = {"N": 64, "K": 128, "nm_n": 0, "nm_m": 0, "codes": P, "meta": None, "alpha": P}
    d.update(kw)
    return bl._Weights(*d.values())


CALLS = {
    "layernorm": [("x", P), ("ldx", 128), ("M", 4), ("K", 128), ("w", P), ("b", P), ("eps", 1e-5), ("y", P),
                  ("mean", P), ("rstd", P), ("stream", None)],
    "layernorm_quant_act": [("x", P), ("ldx", 128), ("M", 4), ("K", 128), ("w", P), ("b", None), ("eps", 1e-5),
                            ("q", P), ("gamma", P), ("rowsum", P), ("mean", None), ("rstd", None), ("stream", None)],
    "layernorm_backward": [("dy", P), ("lddy", 128), ("x", P), ("ldx", 128), ("M", 4), ("K", 128), ("w", P),
                           ("mean", P), ("rstd", P), ("dx", P), ("dw", P), ("db", P), ("workspace", P),
                           ("bytes", 1 << 30), ("stream", None)],
    "rmsnorm_backward": [("dy", P), ("lddy", 128), ("x", P), ("ldx", 128), ("M", 4), ("K", 128), ("g", P),
                         ("eps", 1e-5), ("dx", P), ("dg", P), ("workspace", P), ("bytes", 1 << 30),
                         ("stream", None)],
    "dequant_act": [("q", P), ("ldq", 128), ("gamma", P), ("M", 4), ("K", 128), ("y", P), ("stream", None)],
    "relu2_glu_quant_act": [("g", P), ("ldg", 128), ("u", P), ("ldu", 128), ("M", 4), ("N", 128), ("q_g", P),
                            ("gamma_g", P), ("q_u", P), ("gamma_u", P), ("q_h", P), ("gamma_h", P), ("rowsum_h", P),
                            ("stream", None)],
    "relu2_glu_backward": [("dh", P), ("lddh", 128), ("q_g", P), ("gamma_g", P), ("q_u", P), ("gamma_u", P), ("M", 4),
                           ("N", 128), ("dg", P), ("du", P), ("stream", None)],
    "backward_weight": [("dy", P), ("lddy", 64), ("q", P), ("ldq", 128), ("gamma", P), ("M", 4), ("N", 64),
                        ("K", 128), ("dW", P), ("workspace", P), ("bytes", 1 << 30), ("flags", 0), ("stream", None)],
}
OPTIONAL = {"b", "mean", "rstd", "rowsum", "rowsum_h", "db", "stream", "workspace"}
REQUIRED_STATS = {"layernorm_backward": {"mean", "rstd"}}


def _call(L, name, **kw):
    args = dict(CALLS[name])
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(L, "bitlinear_" + name)(*args.values())


@pytest.mark.parametrize("name", sorted(CALLS))
def test_null_pointers(L, name):
    for arg, v in CALLS[name]:
        if v == P and (arg not in OPTIONAL or arg in REQUIRED_STATS.get(name, ())):
            assert _call(L, name, **{arg: None}) == NULL, arg


@pytest.mark.parametrize("name", sorted(CALLS))
def test_shapes(L, name):
    for arg, v in CALLS[name]:
        if arg in ("M", "N", "K"):
            for bad in (0, -1, (1 << 24) + 1):
                assert _call(L, name, **{arg: bad}) == SHAPE, (arg, bad)
        elif arg.startswith("ld"):
            assert _call(L, name, **{arg: v - 1}) == SHAPE, arg
        elif arg == "eps":
            for bad in (-1e-5, 1.5, float("nan")):
                assert _call(L, name, eps=bad) == SHAPE, bad


@pytest.mark.parametrize("name", sorted(CALLS))
def test_alignment(L, name):
    bytes1 = {"q", "q_g", "q_u", "q_h", "workspace"}
    for arg, v in CALLS[name]:
        if v == P and arg not in bytes1:
            assert _call(L, name, **{arg: P + 1}) == ALIGN, arg


def test_flags(L):
    for bad in (0x1, 0x80, 0x41):
        assert _call(L, "backward_weight", flags=bad) == FLAGS


def test_backward_input(L):
    def call(w, dy=P, lddy=64, M=4, add=None, dx=P):
        return L.bitlinear_backward_input(None if w is None else ctypes.byref(w), dy, lddy, M, add, dx, P, 1 << 30,
                                          None)
    assert call(None) == NULL and call(_weights(), dy=None) == NULL and call(_weights(), dx=None) == NULL
    assert call(_weights(codes=None)) == NULL and call(_weights(nm_n=2, nm_m=4)) == NULL
    assert call(_weights(nm_n=3, nm_m=4, meta=P)) == PATTERN
    assert call(_weights(nm_n=2, nm_m=4, meta=P, K=130)) == SHAPE
    assert call(_weights(), M=0) == SHAPE and call(_weights(), lddy=63) == SHAPE and call(_weights(K=0)) == SHAPE
    assert call(_weights(), dy=P + 1) == ALIGN and call(_weights(), add=P + 1) == ALIGN
    assert call(_weights(), dx=P + 1) == ALIGN and call(_weights(codes=P + 8)) == ALIGN


def test_python_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import ternary_weight_linear_fwd_b200 as bl
    x, w, m = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64), torch.ones(4)
    q = torch.zeros(4, 64, dtype=torch.int8)
    pw = bl.PackedWeights(64, 64, 0, 0, torch.zeros(64, 16, dtype=torch.uint8), None, torch.ones(1))
    for f in (lambda: bl.layernorm(x, w), lambda: bl.layernorm_quant_act(x, w),
              lambda: bl.layernorm_backward(x, x, w, m, m), lambda: bl.rmsnorm_backward(x, x, w, 1e-5),
              lambda: bl.dequant_act(q, m), lambda: bl.relu2_glu_quant_act(x, x),
              lambda: bl.relu2_glu_backward(x, q, m, q, m), lambda: bl.backward_weight(x, q, m),
              lambda: bl.backward_input(pw, x)):
        with pytest.raises(ValueError):
            f()
