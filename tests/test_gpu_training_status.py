"""The gradient products give up on a wait that runs out: status word set, no output, context usable (test build).

As in the other status-word tests the copies all land, but their barrier is told to expect more bytes and the limit
of every wait is cut to milliseconds.  The sizes leave no tile split, whose parts another launch would add up: 6 tiles
and 3 of one k-block each, and 8 x 37 tiles, four whole rounds of 74 pairs."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import ternary_weight_linear_fwd_b200 as bl  # noqa: E402

DEV = torch.device("cuda:0")
PRODUCT_WAIT_NS, SHORT_WAIT_NS = 1_000_000_000, 2_000_000


@pytest.fixture()
def T(monkeypatch):
    """The package bound to the test build of the library."""
    from ternary_weight_linear_fwd_b200 import build as b
    monkeypatch.setattr(bl, "_LIB_PATH", b.build_test_hooks())
    monkeypatch.setattr(bl, "_lib", None)
    bl._workspace_bytes.cache_clear()
    L = bl.lib()
    fn = L.bitlinear_test_set_wait_fault
    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_uint64, ctypes.c_uint32]
    yield L
    assert fn(PRODUCT_WAIT_NS, 0) == 0


@pytest.mark.parametrize("kind,M,N,K", [("weight", 64, 300, 520), ("weight", 1280, 2048, 9472), ("input", 700, 64, 200)])
def test_products_give_up_and_recover(T, kind, M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M)
    dy = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
    q = torch.randint(-127, 128, (M, K), device=DEV, generator=g, dtype=torch.int8)
    gamma = torch.ones(M, device=DEV)
    w = bl.pack_ternary(torch.randint(-1, 2, (N, K), device=DEV, generator=g, dtype=torch.int8), 0.5)
    shape, dtype = ((N, K), torch.float32) if kind == "weight" else ((M, K), torch.bfloat16)

    def call():
        out = torch.full(shape, 12345.0, dtype=dtype, device=DEV)
        bl.backward_weight(dy, q, gamma, out=out) if kind == "weight" else bl.backward_input(w, dy, out=out)
        torch.cuda.synchronize()
        return out

    want = call()
    assert bl.device_status() == 0
    assert T.bitlinear_test_set_wait_fault(SHORT_WAIT_NS, 16) == 0
    got = call()
    assert bl.device_status() in (1, 2, 3, 4, 5)
    assert bool((got == torch.full((), 12345.0, dtype=dtype, device=DEV)).all())
    assert T.bitlinear_test_set_wait_fault(PRODUCT_WAIT_NS, 0) == 0
    assert torch.equal(call(), want) and bl.device_status() == 0
