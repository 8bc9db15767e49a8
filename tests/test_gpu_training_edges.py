"""BitLinear's training side on the GPU where values leave the ordinary range, against plain forms in 64 bits.

Tolerances are those of test_gpu_training.py, with what is added derived beside each check."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import ternary_weight_linear_fwd_b200 as bl  # noqa: E402
from test_gpu_training import BF, DEV, HALF, U, _close, _gen, _norm_backward_ref, _rand, _strided  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ternary_weight_linear_fwd_b200 import build as b
    b.build()
    yield
    torch.cuda.synchronize()
    assert bl.device_status() == 0


# ---------------------------------------------------------------- RMSNorm: rows whose squares fp32 cannot add up
@pytest.mark.parametrize("K", [9, 203, 2560, 6150, 11008, 12290, 16384])
@pytest.mark.parametrize("eps", [1e-5, 0.0])
def test_rmsnorm_backward_far_rows(K, eps):
    """Rows of entries near 1e18 to 3e38, whose squares overflow, and, where no eps hides them, of entries near 1e-25 to
    1e-37, whose squares vanish, among ordinary ones: each row's gradient is that of the formula."""
    M = 40
    x = torch.randn(M, K, device=DEV, generator=_gen(K)).clamp(-4, 4)
    far = {1: 1e17, 4: 1e18, 7: 3e19, 20: 1e25, 21: 1e36, 39: 8e37}
    if eps == 0.0:
        far.update({2: 1e-18, 5: 1e-21, 11: 1e-25, 30: 1e-37})
    for row, scale in far.items():
        x[row] *= scale
    x = x.to(BF)
    assert bool(torch.isfinite(x.float()).all())
    dy = _rand(K + 1, M, K, scale=1e-3)
    g = 1 + 0.1 * torch.randn(K, device=DEV, generator=_gen(1))
    dx, dg = bl.rmsnorm_backward(dy, x, g, eps)
    r = 1.0 / torch.sqrt((x.double() ** 2).mean(1) + float(np.float32(eps)))
    dx0, dg0, _, size, dgs, _ = _norm_backward_ref(dy, x, g, None, r, K)
    # r near the bottom of fp32 is off by half its last place, 2^-150, once in xh and once in front; a result there by
    # half of bf16's, 2^-134
    tiny = 2.0 ** -150 / r[:, None]
    _close(dx, dx0, HALF * dx0.abs() * (1 + HALF) + (256 * U + 3 * tiny) * size + 2.0 ** -134, "dx")
    _close(dg, dg0, ((M + 300) * U + float(tiny.max())) * dgs, "dg")
    for got, want in zip(bl.rmsnorm_backward(_strided(dy, 3, 1), _strided(x, 5, 1), g, eps), (dx, dg)):
        assert torch.equal(got, want)
    # ordinary rows give the bits that they give alone
    keep = torch.tensor([i for i in range(M) if i not in far], device=DEV)
    assert torch.equal(dx[keep], bl.rmsnorm_backward(dy[keep], x[keep], g, eps)[0])


# ---------------------------------------------------------------- layer norm: rows that are constant, or nearly
@pytest.mark.parametrize("K", [7, 203, 641, 2560, 2561, 11008, 16384, 65536])
def test_layernorm_nearly_constant_rows(K):
    """The variance of rows whose mean is far larger than their deviation, as the definition gives it: exactly 0 where all
    entries are equal, whatever they are, and to the last places where one entry (the first, the last, one between) is
    a bf16 step away."""
    fills = [1e4, -1e6, 3e8, 7.7e15, -1e30, 3e38]
    rows = []
    for f in fills:
        base = torch.full((K,), f, device=DEV).to(BF)
        for at in (None, 0, K // 2, K - 1):
            r = base.clone()
            if at is not None:
                r[at] = (base[at].float() * (1 + 2.0 ** -6)).to(BF) if f < 1e38 else (base[at].float() * 0.5).to(BF)
            rows.append(r)
    x = torch.cat([torch.stack(rows), _rand(K, 3, K)])
    w, b = torch.rand(K, device=DEV) + 0.5, torch.rand(K, device=DEV)
    d = x.double()
    mean64 = d[:, :1] + (d - d[:, :1]).mean(1, keepdim=True)
    var = ((d - mean64) ** 2).mean(1).float()  # rounded once, as defined (infinite beyond fp32)
    want = (1.0 / torch.sqrt(var.double() + float(np.float32(1e-5)))).float()
    for xs in (x, _strided(x, 3, 1)):
        y, mean, rstd = bl.layernorm(xs, w, b, 1e-5, want_stats=True)
        q, gamma, _, mean_q, rstd_q = bl.layernorm_quant_act(xs, w, b, 1e-5, want_stats=True)
        assert torch.equal(mean, mean_q) and torch.equal(rstd, rstd_q)
        const = torch.arange(0, 4 * len(fills), 4, device=DEV)
        assert torch.equal(mean[const], x[const, 0].float()) and torch.equal(y[const], b.to(BF).expand(len(fills), K))
        assert torch.equal(rstd[const], want[const])
        # var + eps and the root: the sums in 64 bits leave at most the other neighbour of each fp32 rounding
        _close(rstd, want.double(), 4 * U * want.double(), "rstd")
        m = mean64[:, 0]
        _close(mean, m, U * m.abs() * (1 + 1e-6), "mean")


# ---------------------------------------------------------------- gated FFN: a NaN or an infinity does not vanish
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("N", [1, 16, 203, 272, 6912])
@pytest.mark.parametrize("at", [0, -1])
def test_gate_keeps_what_is_not_a_number(N, at, bad):
    """A gate row with a NaN or an infinity has no restored values: all its gradients are NaN; a row of u, its dg.  Through
    max(., 0) the plain form gives the same.  Other rows keep their bits, on every path."""
    M = 7
    g, u, dh = _rand(N, M, N), _rand(N + 1, M, N), _rand(N + 2, M, N)
    clean = bl.relu2_glu_quant_act(g, u)
    dg0, du0 = bl.relu2_glu_backward(dh, *clean[:4])
    g2, u2 = g.clone(), u.clone()
    g2[2, at] = bad
    u2[4, at] = bad
    for gs, us, ds in ((g2, u2, dh), (_strided(g2, 3, 1), _strided(u2, 5), _strided(dh, 3, 1))):
        c = bl.relu2_glu_quant_act(gs, us)
        assert not bool(torch.isfinite(c.gamma_g[2])) and not bool(torch.isfinite(c.gamma_u[4]))
        if bad != float("-inf"):  # max(-inf, 0) = 0
            assert not bool(torch.isfinite(c.gamma_h[2]))
        assert not bool(torch.isfinite(c.gamma_h[4]))  # r u, or 0 times an infinity
        dg, du = bl.relu2_glu_backward(ds, *c[:4])
        assert bool(dg[2].isnan().all()) and bool(du[2].isnan().all()) and bool(dg[4].isnan().all())
        assert torch.equal(du[4], du0[4])
        keep = [0, 1, 3, 5, 6]
        assert torch.equal(dg[keep], dg0[keep]) and torch.equal(du[keep], du0[keep])
        for got, want in zip(c, clean):
            assert torch.equal(got[keep], want[keep])


# ---------------------------------------------------------------- row-strided views wherever a matrix is read
@pytest.mark.parametrize("M", [1, 21])
@pytest.mark.parametrize("pad,off", [(16, 0), (3, 0), (0, 1)])
def test_strided_codes_and_addend(M, pad, off):
    """The codes that relu2_glu_backward reads and the gradient that backward_input adds, as slices of wider matrices,
    with their columns apart, or expanded."""
    N, K = 272, 200
    c = bl.relu2_glu_quant_act(_rand(1, M, N), _rand(2, M, N))
    dh = _rand(3, M, N, scale=1e-3)
    want = bl.relu2_glu_backward(dh, *c[:4])
    both = torch.cat([c.q_g, c.q_u], 1)
    for q_g, q_u in ((_strided(c.q_g, pad, off), _strided(c.q_u, pad + 5, off)), (both[:, :N], both[:, N:]),
                     (c.q_g.t().contiguous().t(), c.q_u.t().contiguous().t())):
        for got, ref in zip(bl.relu2_glu_backward(dh, q_g, c.gamma_g, q_u, c.gamma_u), want):
            assert torch.equal(got, ref)
    w = bl.pack_ternary(torch.randint(-1, 2, (N, K), device=DEV, generator=_gen(3), dtype=torch.int8), 0.02)
    add = _rand(4, M, K)
    ref = bl.backward_input(w, dh, add=add)
    assert torch.equal(bl.backward_input(w, dh, add=_strided(add, pad, off)), ref)
    one = torch.full((1, 1), 0.25, dtype=BF, device=DEV).expand(M, K)
    assert torch.equal(bl.backward_input(w, dh, add=one), bl.backward_input(w, dh, add=one.contiguous()))
    for bad in (add[:, :-1], add.float(), add.cpu(), add.view(-1)):
        with pytest.raises(ValueError):
            bl.backward_input(w, dh, add=bad)
    for bad in (c.q_g[:, :-1], c.q_g.int(), c.q_g.cpu(), c.q_g.view(-1)):
        with pytest.raises(ValueError):
            bl.relu2_glu_backward(dh, bad, c.gamma_g, c.q_u, c.gamma_u)


# ---------------------------------------------------------------- rows hardly above the codes' 1e-5
def test_small_rows_restored_as_documented():
    """Codes are made with gamma + 1e-5 and stand for q gamma / 127: low by 1% at a maximum of 1e-3, 9% at 1e-4, half at
    1e-5, to within half a step of the codes."""
    tops = [1.0, 1e-2, 1e-3, 1e-4, 1e-5, 1e-7]
    N = 640
    x = torch.randn(len(tops), N, device=DEV, generator=_gen(1)).clamp(-1, 1)
    x[:, 0] = 1.0
    x = (x * torch.tensor(tops, device=DEV)[:, None]).to(BF)
    q, gamma, _ = bl.quant_act(x)
    c = bl.relu2_glu_quant_act(x, x)
    assert torch.equal(c.q_g, q) and torch.equal(c.gamma_u, gamma)
    g = gamma.double()[:, None]
    low = g / (g + 1e-5)
    # half a step of the codes, and the bf16 rounding
    _close(bl.dequant_act(q, gamma), x.double() * low, (0.5 + 1e-3) * g / 127 + HALF * x.double().abs() + 1e-38, "restored")
    dh = torch.ones_like(x)
    dg, du = bl.relu2_glu_backward(dh, *c[:4])
    v = (q.double() * (g / 127)).clamp_min(0)
    _close(du, v * v, (HALF * (1 + HALF) + 6 * U) * v * v + 1e-38, "du")
    _close(dg, 2 * v * v, (HALF * (1 + HALF) + 6 * U) * 2 * v * v + 1e-38, "dg")
