"""Gradient products whose tiles are split give up on a wait that runs out without adding up what an earlier call left
in the workspace: status word set, outputs as they were, context usable (test build; as test_gpu_training_status.py)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import ternary_weight_linear_fwd_b200 as bl  # noqa: E402
from test_gpu_training_status import DEV, PRODUCT_WAIT_NS, SHORT_WAIT_NS, T  # noqa: E402, F401


# only split tiles; whole rounds before them; reductions of several pieces; odd widths
@pytest.mark.parametrize("kind,M,N,K", [("weight", 896, 640, 640), ("weight", 2048, 640, 2560),
                                        ("weight", 2048, 641, 643), ("input", 777, 2560, 640),
                                        ("input", 2048, 6912, 2560), ("input", 700, 2563, 641)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_split_products_give_up_and_recover(T, kind, M, N, K, accumulate):  # noqa: F811
    if kind == "input" and accumulate:
        pytest.skip("the weight gradient's flag")
    g = torch.Generator(device=DEV).manual_seed(M)
    dy = torch.randn(M, N, device=DEV, generator=g).to(torch.bfloat16)
    q = torch.randint(-127, 128, (M, K), device=DEV, generator=g, dtype=torch.int8)
    gamma = torch.ones(M, device=DEV)
    w = bl.pack_ternary(torch.randint(-1, 2, (N, K), device=DEV, generator=g, dtype=torch.int8), 0.5)
    shape, dtype = ((N, K), torch.float32) if kind == "weight" else ((M, K), torch.bfloat16)
    need = (bl.backward_weight_workspace_bytes(M, N, K) if kind == "weight"
            else bl.backward_input_workspace_bytes(w, M))
    assert need >= 256 * 256 * 4  # a slab at least
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)

    def call():
        out = torch.full(shape, 12345.0, dtype=dtype, device=DEV)
        if kind == "weight":
            bl.backward_weight(dy, q, gamma, out=out, accumulate=accumulate, workspace=ws)
        else:
            bl.backward_input(w, dy, out=out, workspace=ws)
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
