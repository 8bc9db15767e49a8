"""BitLinear's training side on the GPU (layer norm, the norms' backward passes, the 8-bit checkpoints of the
gated FFN, the two gradient products) against plain forms in 64 bits.

Tolerances.  A bf16 output is rounded once, by at most half a step: 2^-8 of its value.  To that comes the error
of its fp32 arithmetic, bounded beside each check by (number of roundings) * 2^-24 * (the sum of the absolute
terms).  Codes, row maxima, code sums and restored values are defined to the bit and compared so.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import ternary_weight_linear_fwd_b200 as bl  # noqa: E402

DEV = torch.device("cuda:0")
BF = torch.bfloat16
HALF = 2.0 ** -8   # half a bf16 step, relative
U = 2.0 ** -24     # half an fp32 step, relative


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ternary_weight_linear_fwd_b200 import build as b
    b.build()
    yield
    torch.cuda.synchronize()
    assert bl.device_status() == 0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rand(seed, *shape, scale=1.0, outliers=False):
    g = _gen(seed)
    x = scale * torch.randn(*shape, device=DEV, generator=g)
    if outliers:
        x = torch.where(torch.rand(*shape, device=DEV, generator=g) < 0.01, 10 * x, x)
    return x.to(BF)


def _strided(t, pad, off=0):
    """The same values as a view whose rows lie t.shape[1] + pad elements apart, off elements into a buffer."""
    M, K = t.shape
    buf = torch.full((M * (K + pad) + off,), 7, dtype=t.dtype, device=t.device)
    v = buf[off:].view(M, K + pad)[:, :K]
    v.copy_(t)
    return v


def _close(got, want, bound, what):
    """|got - want| <= bound everywhere (want, bound in 64 bits); NaN only where both have it."""
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error / bound "
        f"{float(((got - want).abs() / bound.clamp_min(1e-300)).nan_to_num(float('inf')).max()):.3g}")


# ---------------------------------------------------------------- plain forms
def _moments(x, eps):
    """mean and rstd as the header defines them: sums in 64 bits, each result rounded to fp32 once."""
    d = x.double()
    K = x.shape[1]
    s1, s2 = d.sum(1), (d * d).sum(1)
    mean = (s1 / K).float()
    var = ((s2 - s1 * s1 / K) / K).clamp_min(0).float()
    eps32 = float(np.float32(eps))
    return mean, (1.0 / torch.sqrt(var.double() + eps32)).float()


def _normed(x, w, b, mean, rstd):
    y = (x.float() - mean[:, None]) * rstd[:, None] * w
    return y if b is None else y + b


def _codes(v):
    """quant_act's codes of fp32 rows: (q, gamma, rowsum)."""
    gamma = v.abs().amax(1)
    q = torch.round((v * 127.0) / (gamma + np.float32(1e-5))[:, None]).clamp(-128, 127)
    return q.to(torch.int8), gamma, q.to(torch.int32).sum(1, dtype=torch.int32)


def _values(q, gamma):
    return q.float() * (gamma / 127.0)[:, None]


def _glu_h(g, u):
    return (torch.relu(g.float()).square().to(BF).float() * u.float()).to(BF)


# ---------------------------------------------------------------- layer norm
LN_SHAPES = [(1, 1), (1, 2560), (3, 7), (5, 203), (16, 2560), (33, 640), (257, 2048), (700, 2560), (64, 6912),
             (2, 16384), (3, 12301), (2, 65536)]


@pytest.mark.parametrize("M,K", LN_SHAPES)
@pytest.mark.parametrize("bias", [False, True])
def test_layernorm(M, K, bias):
    x = _rand(M + K, M, K, outliers=True)
    w = 1 + 0.1 * torch.randn(K, device=DEV, generator=_gen(1))
    b = 0.1 * torch.randn(K, device=DEV, generator=_gen(2)) if bias else None
    y, mean, rstd = bl.layernorm(x, w, b, 1e-5, want_stats=True)
    m0, r0 = _moments(x, 1e-5)
    assert torch.equal(mean, m0) and torch.equal(rstd, r0)
    want = ((x.double() - m0.double()[:, None]) * r0.double()[:, None] * w.double()
            + (0.0 if b is None else b.double()))
    # three or four fp32 roundings of terms no larger than |xn| and |b|
    _close(y, want, HALF * want.abs() * (1 + HALF) + 5 * U * (want.abs() + (0 if b is None else b.abs().double())),
           "y")
    assert torch.equal(y, _normed(x, w, b, m0, r0).to(BF))
    q, gamma, rs, mean, rstd = bl.layernorm_quant_act(x, w, b, 1e-5, want_stats=True)
    q0, g0, rs0 = _codes(_normed(x, w, b, m0, r0))
    assert torch.equal(mean, m0) and torch.equal(rstd, r0)
    assert torch.equal(gamma, g0) and torch.equal(q, q0) and torch.equal(rs, rs0)


@pytest.mark.parametrize("fill", [0.0, 3.0, -250.0])
def test_layernorm_constant_rows(fill):
    """A padded (zero) row, and constant ones: variance exactly 0, the output is the bias."""
    M, K = 4, 2560
    x = _rand(5, M, K)
    x[1] = fill
    w, b = torch.ones(K, device=DEV), torch.full((K,), 0.5, device=DEV)
    y, mean, rstd = bl.layernorm(x, w, b, 1e-5, want_stats=True)
    assert float(mean[1]) == fill and torch.equal(y[1], b.to(BF))
    assert float(rstd[1]) == float(np.float32(1.0 / np.sqrt(float(np.float32(1e-5)))))
    q, gamma, _ = bl.layernorm_quant_act(x, w, None, 1e-5)
    assert float(gamma[1]) == 0.0 and not q[1].any()


def test_layernorm_large_mean_small_spread():
    """Mean 200, deviation about 1: the one-pass variance in 64 bits keeps all 24 bits of its result."""
    x = (200 + torch.randn(9, 2560, device=DEV, generator=_gen(3))).to(BF)
    _, mean, rstd = bl.layernorm(x, torch.ones(2560, device=DEV), None, 1e-5, want_stats=True)
    d = x.double()
    assert torch.equal(mean, d.mean(1).float())
    want = 1 / torch.sqrt(d.var(1, unbiased=False) + 1e-5)
    _close(rstd, want, 4 * U * want, "rstd")


@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (0, 1), (8, 4)])
def test_layernorm_strided(pad, off):
    x = _rand(7, 37, 640)
    w, b = torch.rand(640, device=DEV), torch.rand(641, device=DEV)[1:]
    assert torch.equal(bl.layernorm(_strided(x, pad, off), w, b, 1e-6), bl.layernorm(x, w, b, 1e-6))
    for got, want in zip(bl.layernorm_quant_act(_strided(x, pad, off), w, b, 1e-6),
                         bl.layernorm_quant_act(x, w, b, 1e-6)):
        assert torch.equal(got, want)


# ---------------------------------------------------------------- backward of the norms
NB_SHAPES = [(1, 1), (1, 2560), (7, 9), (5, 203), (16, 2560), (333, 640), (1000, 2560), (300, 6144), (41, 6150),
             (150, 11008), (20, 12288), (6, 12290), (70, 16384), (3, 65536)]


def _norm_backward_ref(dy, x, w, mean, rstd, K):
    """dx, dw, db and the sums of absolute terms behind dx and dw, in 64 bits; mean None: RMSNorm."""
    dy, x, w, rstd = dy.double(), x.double(), w.double(), rstd.double()[:, None]
    xh = (x if mean is None else x - mean.double()[:, None]) * rstd
    a = dy * w
    c2 = (a * xh).sum(1, keepdim=True) / K
    c1 = 0.0 if mean is None else a.sum(1, keepdim=True) / K
    dx = rstd * (a - c1 - xh * c2)
    size = rstd * (a.abs() + (0.0 if mean is None else a.abs().sum(1, keepdim=True) / K)
                   + xh.abs() * (a * xh).abs().sum(1, keepdim=True) / K)
    # |x| + |mean| may cancel in x - mean, which is one rounding of the difference: no more than |xh|
    return dx, (dy * xh).sum(0), dy.sum(0), size, (dy * xh).abs().sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("M,K", NB_SHAPES)
def test_layernorm_backward(M, K):
    x, dy = _rand(M * 3 + K, M, K, outliers=True), _rand(M + K * 5, M, K, scale=1e-3)
    if M > 8:
        dy[-(M // 8):] = 0  # padded tokens
    w = 1 + 0.1 * torch.randn(K, device=DEV, generator=_gen(1))
    mean, rstd = _moments(x, 1e-5)
    dx, dw, db = bl.layernorm_backward(dy, x, w, mean, rstd)
    dx0, dw0, db0, size, dws, dbs = _norm_backward_ref(dy, x, w, mean, rstd, K)
    # sums over K: at most 64 terms a thread, 10 levels of lanes and 32 warps, about 10 roundings a term
    _close(dx, dx0, HALF * dx0.abs() * (1 + HALF) + 128 * U * size, "dx")
    # sums over M: every row one rounding, plus those of the term itself and of the partial sums
    _close(dw, dw0, (M + 200) * U * dws, "dw")
    _close(db, db0, (M + 200) * U * dbs, "db")
    again = bl.layernorm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    dx2, dw2, none = bl.layernorm_backward(dy, x, w, mean, rstd, want_bias=False)
    assert none is None and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("M,K", NB_SHAPES)
def test_rmsnorm_backward(M, K):
    x, dy = _rand(M * 5 + K, M, K, outliers=True), _rand(M + K * 7, M, K, scale=1e-3)
    if M > 8:
        x[-(M // 8):] = 0
        dy[-(M // 8):] = 0
    g = 1 + 0.1 * torch.randn(K, device=DEV, generator=_gen(1))
    dx, dg = bl.rmsnorm_backward(dy, x, g, 1e-5)
    rstd = 1.0 / torch.sqrt((x.double() ** 2).mean(1) + float(np.float32(1e-5)))
    dx0, dg0, _, size, dgs, _ = _norm_backward_ref(dy, x, g, None, rstd, K)
    # rstd itself is recomputed: half the 128 roundings of its sum, a root and a quotient
    _close(dx, dx0, HALF * dx0.abs() * (1 + HALF) + 256 * U * size, "dx")
    _close(dg, dg0, (M + 300) * U * dgs, "dg")


@pytest.mark.parametrize("pad,off", [(8, 0), (5, 0), (0, 1)])
def test_norm_backward_strided(pad, off):
    M, K = 45, 1000
    x, dy = _rand(1, M, K), _rand(2, M, K, scale=1e-3)
    w = torch.rand(K, device=DEV)
    mean, rstd = _moments(x, 1e-5)
    for got, want in zip(bl.layernorm_backward(_strided(dy, pad, off), _strided(x, pad + 8, off), w, mean, rstd),
                         bl.layernorm_backward(dy, x, w, mean, rstd)):
        assert torch.equal(got, want)
    for got, want in zip(bl.rmsnorm_backward(_strided(dy, pad + 16, off), _strided(x, pad, off), w, 1e-6),
                         bl.rmsnorm_backward(dy, x, w, 1e-6)):
        assert torch.equal(got, want)


def test_norm_gradients_against_differences():
    """The formulas against central differences of the forward pass in 64 bits, then the kernels against both."""
    M, K, eps, h = 3, 40, 1e-5, 1e-5
    x, dy = _rand(11, M, K), _rand(12, M, K)
    w, b = torch.rand(K, device=DEV) + 0.5, torch.rand(K, device=DEV)

    def loss(kind, xd, wd, bd):
        c = xd - xd.mean(1, keepdim=True) if kind == "layer" else xd
        return ((c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * wd + bd) * dy.double()).sum()

    for kind in ("layer", "rms"):
        args = [x.double(), w.double(), b.double()]
        num = []
        for i, t in enumerate(args):
            d = torch.zeros_like(t).view(-1)
            for j in range(t.numel()):
                two = []
                for sgn in (1, -1):
                    moved = [v.clone() for v in args]
                    moved[i].view(-1)[j] += sgn * h
                    two.append(loss(kind, *moved))
                d[j] = (two[0] - two[1]) / (2 * h)
            num.append(d.view_as(t))
        mean, rstd = _moments(x, eps)
        r64 = 1 / torch.sqrt((x.double() ** 2).mean(1) + eps)
        ref = _norm_backward_ref(dy, x, w, mean if kind == "layer" else None, rstd if kind == "layer" else r64, K)
        for a, n in zip(ref[:3] if kind == "layer" else ref[:2], num):
            # differences of a function of size ~100 with h = 1e-5: 100 * 2^-53 / h + third derivative * h^2
            assert float((a - n).abs().max()) < 1e-5 * max(1.0, float(n.abs().max()))
        got = bl.layernorm_backward(dy, x, w, mean, rstd) if kind == "layer" else bl.rmsnorm_backward(dy, x, w, eps)
        assert float((got[0].double() - num[0]).abs().max()) < HALF * float(num[0].abs().max()) + 1e-4
        assert float((got[1].double() - num[1]).abs().max()) < 1e-4


# ---------------------------------------------------------------- 8-bit checkpoints
GLU_SHAPES = [(1, 1), (1, 6912), (5, 203), (16, 2560), (77, 6912), (300, 640), (9, 11008), (3, 12301), (2, 16384),
              (2, 65536)]


@pytest.mark.parametrize("M,N", GLU_SHAPES)
def test_relu2_glu_checkpoint(M, N):
    g, u = _rand(M + N, M, N, outliers=True), _rand(M * 3 + N, M, N)
    if M > 2:
        g[1] = -g[1].abs()  # h = 0 on the whole row
        g[2] = 0
    c = bl.relu2_glu_quant_act(g, u)
    for v, q, gamma in ((g, c.q_g, c.gamma_g), (u, c.q_u, c.gamma_u), (_glu_h(g, u), c.q_h, c.gamma_h)):
        q0, g0, rs0 = _codes(v.float())
        assert torch.equal(gamma, g0) and torch.equal(q, q0)
    assert torch.equal(c.rowsum_h, rs0)
    # the same codes as the forward's own quantisation, where it reads such rows
    qh, gh, rsh = bl.quant_act(_glu_h(g, u))
    assert torch.equal(c.q_h, qh) and torch.equal(c.gamma_h, gh) and torch.equal(c.rowsum_h, rsh)
    assert torch.equal(bl.dequant_act(c.q_h, c.gamma_h), _values(c.q_h, c.gamma_h).to(BF))

    dh = _rand(M + 2 * N, M, N, scale=1e-3)
    dg, du = bl.relu2_glu_backward(dh, c.q_g, c.gamma_g, c.q_u, c.gamma_u)
    gv, uv, d = (t.double() for t in (_values(c.q_g, c.gamma_g), _values(c.q_u, c.gamma_u), dh))
    r = torch.relu(gv)
    # two products and the value's own rounding: at most 4 fp32 roundings
    _close(dg, 2 * d * r * uv, (HALF * (1 + HALF) + 4 * U) * (2 * d * r * uv).abs() + 1e-38, "dg")
    _close(du, d * r * r, (HALF * (1 + HALF) + 4 * U) * (d * r * r).abs() + 1e-38, "du")


def test_relu2_glu_gradient_against_differences():
    """dg, du at the checkpointed values are the differences of h = max(g, 0)^2 u there."""
    g, u, dh = _rand(1, 4, 64), _rand(2, 4, 64), _rand(3, 4, 64)
    c = bl.relu2_glu_quant_act(g, u)
    dg, du = bl.relu2_glu_backward(dh, c.q_g, c.gamma_g, c.q_u, c.gamma_u)
    gv, uv = _values(c.q_g, c.gamma_g).double(), _values(c.q_u, c.gamma_u).double()
    f = lambda a, b: torch.relu(a) ** 2 * b * dh.double()  # noqa: E731
    h = 1e-6
    ng = (f(gv + h, uv) - f(gv - h, uv)) / (2 * h)
    nu = (f(gv, uv + h) - f(gv, uv - h)) / (2 * h)
    # central differences of a piecewise quadratic: exact but for 1e-16 / h and, at the kink, h |u dh|
    _close(dg, ng, HALF * 1.01 * ng.abs() + 1e-4, "dg")
    _close(du, nu, HALF * 1.01 * nu.abs() + 1e-4, "du")


@pytest.mark.parametrize("pad,off", [(16, 0), (3, 0), (0, 1)])
def test_checkpoint_strided(pad, off):
    M, N = 21, 272
    g, u, dh = _rand(1, M, N), _rand(2, M, N), _rand(3, M, N, scale=1e-3)
    c = bl.relu2_glu_quant_act(g, u)
    for a, b in zip(bl.relu2_glu_quant_act(_strided(g, pad, off), _strided(u, pad + 8, off)), c):
        assert torch.equal(a, b)
    args = (c.q_g, c.gamma_g, c.q_u, c.gamma_u)
    for a, b in zip(bl.relu2_glu_backward(_strided(dh, pad, off), *args), bl.relu2_glu_backward(dh, *args)):
        assert torch.equal(a, b)
    assert torch.equal(bl.dequant_act(_strided(c.q_h, pad, off), c.gamma_h), bl.dequant_act(c.q_h, c.gamma_h))
    # both halves of one gate-and-up output, as a fused projection writes them
    gu = torch.cat([g, u], 1)
    for a, b in zip(bl.relu2_glu_quant_act(gu[:, :N], gu[:, N:]), c):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- gradient products
GEMM_SHAPES = [(1, 1, 1), (1, 2560, 640), (2, 9, 17), (16, 640, 2560), (63, 65, 127), (64, 64, 64), (65, 63, 129),
               (100, 203, 301), (128, 256, 256), (255, 257, 511), (256, 512, 256), (257, 130, 1000),
               (300, 2560, 2560), (777, 640, 2560), (2048, 640, 1024), (33, 6912, 200), (1000, 72, 4104),
               (5000, 96, 160), (1, 20000, 8), (40, 8, 40000)]


def _checkpoint(seed, M, K):
    x = _rand(seed, M, K, outliers=True)
    if M > 3:
        x[M // 2] = 0
    q, gamma, _ = _codes(x.float())
    return q, gamma


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_backward_weight(M, N, K):
    dy = _rand(M + N, M, N, scale=1e-3)
    q, gamma = _checkpoint(M + K, M, K)
    dW = bl.backward_weight(dy, q, gamma)
    x = _values(q, gamma).to(BF).double()
    want, size = dy.double().t() @ x, dy.double().abs().t() @ x.abs()
    # the products are exact; M additions, each off by at most one fp32 step (the tensor cores truncate)
    bound = 2 * (M + 16) * U * size
    _close(dW, want, bound, "dW")
    assert torch.equal(dW, bl.backward_weight(dy, q, gamma))
    acc = torch.randn(N, K, device=DEV, generator=_gen(4)) * 1e-3
    out = acc.clone()
    assert bl.backward_weight(dy, q, gamma, out=out, accumulate=True).data_ptr() == out.data_ptr()
    _close(out, want + acc.double(), bound + 2 * (M // 256 + 2) * U * (acc.abs().double() + size), "dW accumulated")


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_backward_input_dense(M, N, K, add):
    T = torch.randint(-1, 2, (N, K), device=DEV, generator=_gen(N + K), dtype=torch.int8)
    w = bl.pack_ternary(T, 0.037)
    _check_input(w, T, _rand(M + N, M, N, scale=1e-3), _rand(M, M, K, scale=1e-3) if add else None)


def _check_input(w, T, dy, add):
    dx = bl.backward_input(w, dy, add=add)
    alpha = float(w.alpha)
    s = dy.double() @ T.double() * alpha
    size = dy.double().abs() @ T.double().abs() * alpha
    want = s if add is None else s + add.double()
    N = w.N
    # exact products, N additions off by at most one fp32 step each, the scale and the sum one rounding each
    _close(dx, want, HALF * 1.01 * want.abs() + 2 * (N + 16) * U * (size + (0 if add is None else add.abs().double())),
           "dx")
    assert torch.equal(dx, bl.backward_input(w, dy, add=add))


@pytest.mark.parametrize("n,m", [(2, 4), (1, 8), (3, 8), (4, 8), (6, 8), (7, 8)])
@pytest.mark.parametrize("M,N,K", [(1, 33, 8), (70, 130, 264), (300, 640, 2560), (257, 96, 1032)])
def test_backward_input_nm(n, m, M, N, K):
    W = 0.02 * torch.randn(N, K, device=DEV, generator=_gen(n * m))
    w = bl.pack_weights(W, n, m)
    blocks = W.view(N, K // m, m)
    keep = torch.zeros_like(blocks).scatter_(2, blocks.abs().argsort(dim=2, descending=True, stable=True)[:, :, :n], 1)
    T = (torch.round(W / (w.alpha + 1e-5)).clamp(-1, 1) * keep.view(N, K)).to(torch.int8)
    _check_input(w, T, _rand(M + N, M, N, scale=1e-3), _rand(M, M, K, scale=1e-3))


@pytest.mark.parametrize("pad,off", [(8, 0), (16, 8), (3, 0), (0, 1), (13, 5)])
def test_gradient_products_strided(pad, off):
    M, N, K = 150, 264, 272
    dy = _rand(1, M, N, scale=1e-3)
    q, gamma = _checkpoint(2, M, K)
    T = torch.randint(-1, 2, (N, K), device=DEV, generator=_gen(3), dtype=torch.int8)
    w = bl.pack_ternary(T, 0.02)
    assert torch.equal(bl.backward_weight(_strided(dy, pad, off), _strided(q, 2 * pad, 2 * off), gamma),
                       bl.backward_weight(dy, q, gamma))
    assert torch.equal(bl.backward_input(w, _strided(dy, pad, off)), bl.backward_input(w, dy))
    # the gradient of a mean: an expanded tensor, all strides 0
    one = torch.full((1, 1), 1e-3, dtype=BF, device=DEV).expand(M, N)
    assert torch.equal(bl.backward_input(w, one), bl.backward_input(w, one.contiguous()))
    assert torch.equal(bl.backward_weight(one, q, gamma), bl.backward_weight(one.contiguous(), q, gamma))
    # column-major gradients are copied
    assert torch.equal(bl.backward_input(w, dy.t().contiguous().t()), bl.backward_input(w, dy))


def test_gradient_products_leave_padding_and_neighbours():
    """Outputs of odd sizes end inside tiles: nothing outside them is written."""
    M, N, K = 77, 45, 83
    dy = _rand(1, M, N)
    q, gamma = _checkpoint(2, M, K)
    w = bl.pack_ternary(torch.randint(-1, 2, (N, K), device=DEV, dtype=torch.int8, generator=_gen(1)), 0.1)
    buf = torch.full((N * K + 512,), 3.0, device=DEV)
    bl.backward_weight(dy, q, gamma, out=buf[256:256 + N * K].view(N, K))
    assert bool((buf[:256] == 3).all()) and bool((buf[256 + N * K:] == 3).all())
    bufx = torch.full((M * K + 512,), 3.0, device=DEV, dtype=BF)
    bl.backward_input(w, dy, out=bufx[256:256 + M * K].view(M, K))
    assert bool((bufx[:256] == 3).all()) and bool((bufx[256 + M * K:] == 3).all())


def test_straight_through_gradient():
    """The products are the gradients that autograd finds through the two straight-through quantisers."""
    M, N, K = 24, 40, 56
    W = (0.02 * torch.randn(N, K, device=DEV, generator=_gen(1))).requires_grad_()
    x = _rand(2, M, K).float().requires_grad_()
    dy = _rand(3, M, N, scale=1e-2)
    w = bl.pack_weights(W.detach())
    q, gamma, _ = bl.quant_act(x.detach().to(BF))
    Wq = torch.round(W.detach() / (w.alpha + 1e-5)).clamp(-1, 1) * w.alpha
    xq = bl.dequant_act(q, gamma).float()
    y = (x + (xq - x).detach()) @ (W + (Wq - W).detach()).t()
    y.backward(dy.float())
    size = float(x.grad.abs().max())
    assert float((bl.backward_input(w, dy).float() - x.grad).abs().max()) < (HALF + 1e-5) * size
    assert float((bl.backward_weight(dy, q, gamma) - W.grad).abs().max()) < 1e-5 * float(W.grad.abs().max())


# ---------------------------------------------------------------- far offsets
def test_offsets_beyond_31_bits():
    """More than 2^31 elements: the last rows are computed as they are alone."""
    M, K = 33000, 65536
    x = torch.empty((M, K), dtype=BF, device=DEV)
    x[:8] = _rand(1, 8, K)
    x[8:] = x[:8].repeat((M - 8 + 7) // 8, 1)[:M - 8]
    last = x[-8:].contiguous()
    w = torch.rand(K, device=DEV) + 0.5
    q, gamma, rs, mean, rstd = bl.layernorm_quant_act(x, w, None, 1e-5, want_stats=True)
    for got, want in zip((q, gamma, rs), bl.layernorm_quant_act(last, w, None, 1e-5)):
        assert torch.equal(got[-8:], want)
    y = bl.dequant_act(q, gamma)
    assert torch.equal(y[-8:], bl.dequant_act(q[-8:].contiguous(), gamma[-8:].contiguous()))
    del y
    dx, _, _ = bl.layernorm_backward(x, x, w, mean, rstd)
    want, _, _ = bl.layernorm_backward(last, last, w, mean[-8:].contiguous(), rstd[-8:].contiguous())
    assert torch.equal(dx[-8:], want)
    del dx
    # gradient products whose dx and q pass 2^31 elements
    N = 64
    pw = bl.pack_ternary(torch.randint(-1, 2, (N, K), device=DEV, dtype=torch.int8, generator=_gen(5)), 0.02)
    dy = x[:, :N].contiguous()
    dx = bl.backward_input(pw, dy)
    T = bl.backward_input(pw, dy[-8:].contiguous())
    assert float((dx[-8:].float() - T.float()).abs().max()) <= HALF * 2 * float(T.float().abs().max())
    del dx
    only = torch.zeros_like(dy)
    only[-8:] = dy[-8:]
    a, b = bl.backward_weight(only, q, gamma), bl.backward_weight(dy[-8:].contiguous(), q[-8:].contiguous(),
                                                                  gamma[-8:].contiguous())
    assert float((a - b).abs().max()) <= 64 * U * float(b.abs().max())


# ---------------------------------------------------------------- together, streams, graphs
def _ffn_step(x, dy, lw, lb, wg, wu, wd):
    """Forward and backward pass of layer norm -> gate/up -> squared-ReLU gate -> down, as a program runs it."""
    q, gamma, rs, mean, rstd = bl.layernorm_quant_act(x, lw, lb, 1e-5, want_stats=True)
    g, u = bl.forward_q8(wg, q, gamma, rs), bl.forward_q8(wu, q, gamma, rs)
    c = bl.relu2_glu_quant_act(g, u)
    y = bl.forward_q8(wd, c.q_h, c.gamma_h, c.rowsum_h)
    dwd = bl.backward_weight(dy, c.q_h, c.gamma_h)
    dh = bl.backward_input(wd, dy)
    dg, du = bl.relu2_glu_backward(dh, c.q_g, c.gamma_g, c.q_u, c.gamma_u)
    dwg, dwu = bl.backward_weight(dg, q, gamma), bl.backward_weight(du, q, gamma)
    dxn = bl.backward_input(wu, du, add=bl.backward_input(wg, dg))
    dx, dlw, dlb = bl.layernorm_backward(dxn, x, lw, mean, rstd)
    return y, dx, dlw, dlb, dwg, dwu, dwd


def _ffn_plain(x, dy, lw, lb, wg, wu, wd):
    """The same step in 64 bits between the roundings that the calls define."""
    mean, rstd = _moments(x, 1e-5)
    q, gamma, _ = _codes(_normed(x, lw, lb, mean, rstd))
    xt = _values(q, gamma).to(BF).double()
    mats = []
    for w in (wg, wu, wd):
        shift = torch.arange(0, 8, 2, device=DEV, dtype=torch.int32)
        T = ((w.codes.int()[:, :, None] >> shift) & 3).view(w.N, -1)[:, :w.K].double() - 1
        mats.append(T)
    lin = lambda q, gamma, T, w: ((q.double() @ T.t()).float() * (w.alpha * gamma / 127.0)[:, None]).to(BF)  # noqa: E731
    g, u = lin(q, gamma, mats[0], wg), lin(q, gamma, mats[1], wu)
    h = _glu_h(g, u)
    qg, gg, _ = _codes(g.float())
    qu, gu, _ = _codes(u.float())
    qh, gh, _ = _codes(h.float())
    y = lin(qh, gh, mats[2], wd)
    al = [w.alpha.double() for w in (wg, wu, wd)]
    ht = _values(qh, gh).to(BF).double()
    dwd = dy.double().t() @ ht
    dh = dy.double() @ mats[2] * al[2]
    r, uv = torch.relu(_values(qg, gg).double()), _values(qu, gu).double()
    dg, du = 2 * dh * r * uv, dh * r * r
    dxn = dg @ mats[0] * al[0] + du @ mats[1] * al[1]
    ref = _norm_backward_ref(dxn, x, lw, mean, rstd, x.shape[1])
    return y, ref[0], ref[1], ref[2], dg.t() @ xt, du.t() @ xt, dwd


def _ffn_inputs(M=200, D=256, F=640, seed=0):
    mk = lambda s, n, k: bl.pack_ternary(  # noqa: E731
        torch.randint(-1, 2, (n, k), device=DEV, generator=_gen(seed + s), dtype=torch.int8), 0.03)
    return (_rand(seed + 1, M, D, outliers=True), _rand(seed + 2, M, D, scale=1e-3),
            1 + 0.1 * torch.randn(D, device=DEV, generator=_gen(seed + 3)),
            0.1 * torch.randn(D, device=DEV, generator=_gen(seed + 4)), mk(5, F, D), mk(6, F, D), mk(7, D, F))


def test_ffn_step():
    """One training step through all of it.  Between dy and the last gradient lie at most four bf16 roundings
    (dh; dg, du; the first summand of dxn; dxn), each of at most 2^-8 of its tensor's norm: 2^-6 in all."""
    args = _ffn_inputs()
    got, want = _ffn_step(*args), _ffn_plain(*args)
    assert torch.equal(got[0], want[0])
    for name, a, b in zip(("dx", "dlw", "dlb", "dWg", "dWu", "dWd"), got[1:], want[1:]):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < 2.0 ** -6, (name, rel)


def test_ffn_step_captured_and_replayed():
    """The step captured into a graph gives the eager bits, again for new inputs copied in place, and while an
    eager run of the same tensors lives beside it; a second graph shares nothing with the first."""
    a, b = _ffn_inputs(seed=0), _ffn_inputs(seed=100)
    eager_a, eager_b = _ffn_step(*a), _ffn_step(*b)
    x, dy = a[0].clone(), a[1].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _ffn_step(x, dy, *a[2:])
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _ffn_step(x, dy, *a[2:])
        graphs.append((g, out))
    for g, out in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(p, q) for p, q in zip(out, eager_a))
    x.copy_(b[0])
    dy.copy_(b[1])
    mixed = _ffn_step(b[0], b[1], *a[2:])
    # the two graphs at once on two streams
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    graphs[0][0].replay()
    with torch.cuda.stream(s2):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(p, q) for p, q in zip(out, mixed))
    del eager_b


def test_two_streams_at_once():
    """Calls on two streams at the same time, each with workspaces of its own."""
    a, b = _ffn_inputs(seed=0), _ffn_inputs(seed=50)
    want = _ffn_step(*a), _ffn_step(*b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (s, args) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i].append(_ffn_step(*args))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(run, want[i]))


def test_stream_argument():
    x, dy, lw, lb, wg, wu, wd = _ffn_inputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bl.backward_input(wg, _rand(9, 200, 640), stream=s)
    q, gamma, _ = bl.layernorm_quant_act(x, lw, lb, 1e-5, stream=s)
    dW = bl.backward_weight(dy, q, gamma, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, bl.backward_input(wg, _rand(9, 200, 640)))
    assert torch.equal(dW, bl.backward_weight(dy, q, gamma))


# ---------------------------------------------------------------- refusals
def test_refusals():
    x = _rand(1, 8, 64)
    w = torch.ones(64, device=DEV)
    q, gamma, _ = bl.quant_act(x)
    mean, rstd = _moments(x, 1e-5)
    pw = bl.pack_ternary(torch.zeros(32, 64, dtype=torch.int8, device=DEV), 1.0)
    dy = _rand(2, 8, 32)
    refused = [
        lambda: bl.layernorm(x.float(), w), lambda: bl.layernorm(x[0], w), lambda: bl.layernorm(x, w[:63]),
        lambda: bl.layernorm(x, w.to(BF)), lambda: bl.layernorm(x, w, w.cpu()),
        lambda: bl.layernorm(x, w, out=torch.empty(8, 63, dtype=BF, device=DEV)),
        lambda: bl.layernorm_backward(dy, x, w, mean, rstd), lambda: bl.layernorm_backward(x, x, w, mean[:7], rstd),
        lambda: bl.layernorm_backward(x, x, w, mean, rstd, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
        lambda: bl.rmsnorm_backward(x, x.float(), w, 1e-5),
        lambda: bl.dequant_act(x, gamma), lambda: bl.dequant_act(q, gamma[:7]),
        lambda: bl.relu2_glu_quant_act(x, dy), lambda: bl.relu2_glu_backward(x, q[:, :32], gamma, q, gamma),
        lambda: bl.relu2_glu_backward(x, q, gamma.int(), q, gamma),
        lambda: bl.backward_weight(dy[:7], q, gamma), lambda: bl.backward_weight(dy, q.int(), gamma),
        lambda: bl.backward_weight(dy, q, gamma, accumulate=True),
        lambda: bl.backward_weight(dy, q, gamma, out=torch.empty(32, 64, device=DEV, dtype=BF)),
        lambda: bl.backward_input(pw, x), lambda: bl.backward_input(pw, dy.float()),
        lambda: bl.backward_input(pw, dy, add=dy),
    ]
    for f in refused:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: bl.layernorm(x, w, eps=-1.0), lambda: bl.layernorm(x, w, eps=float("nan")),
              lambda: bl.layernorm(x[:0], w), lambda: bl.rmsnorm_backward(x, x, w, 2.0),
              lambda: bl.layernorm_backward(x, x, w, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8,
                                                                                       device=DEV)),
              lambda: bl.backward_weight(dy[:0], q[:0], gamma[:0]), lambda: bl.backward_input(pw, dy[:0])):
        with pytest.raises(bl.BitLinearError):
            f()


# ---------------------------------------------------------------- products large enough to restore an operand first
@pytest.mark.parametrize("M,N,K", [(4096, 2600, 2100), (2200, 6912, 2563), (8000, 1300, 1500)])
def test_backward_weight_restored_operand(M, N, K):
    dy = _rand(M + N, M, N, scale=1e-3)
    dy[-M // 8:] = 0
    q, gamma = _checkpoint(M + K, M, K)
    x = _values(q, gamma).to(BF)
    want, size = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    dW = bl.backward_weight(dy, q, gamma)
    _close(dW, want, 2 * (M + 16) * U * size, "dW")
    # a strided checkpoint of odd width, and a second run, give the same bits
    assert torch.equal(dW, bl.backward_weight(_strided(dy, 8), _strided(q, 13), gamma))
    out = torch.ones(N, K, device=DEV)
    bl.backward_weight(dy, q, gamma, out=out, accumulate=True)
    _close(out, want + 1, 2 * (M + 16) * U * size + 2 * (M // 256 + 2) * U * (1 + size), "dW accumulated")


@pytest.mark.parametrize("n,m", [(0, 0), (2, 4), (3, 8)])
@pytest.mark.parametrize("M,N,K", [(4100, 8200, 2056), (16000, 1000, 2568)])
def test_backward_input_restored_operand(n, m, M, N, K):
    W = 0.02 * torch.randn(N, K, device=DEV, generator=_gen(n * m))
    w = bl.pack_weights(W, n, m)
    T = torch.round(W / (w.alpha + 1e-5)).clamp(-1, 1)
    if m:
        blocks = W.view(N, K // m, m)
        T *= torch.zeros_like(blocks).scatter_(2, blocks.abs().argsort(dim=2, descending=True, stable=True)[:, :, :n],
                                               1).view(N, K)
    _check_input(w, T.to(torch.int8), _rand(M + N, M, N, scale=1e-3), _rand(M, M, K, scale=1e-3))


# ---------------------------------------------------------------- rows that are not numbers
@pytest.mark.parametrize("K", [16, 203, 2560, 11008])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_layernorm_keeps_nan(K, bad):
    """A row with a NaN or an infinity has no mean: its output, row maximum and restored values are NaN; others stay."""
    x = _rand(K, 9, K)
    y = x.clone()
    y[4, K // 2] = bad
    w, b = torch.rand(K, device=DEV) + 0.5, torch.rand(K, device=DEV)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    out, clean = bl.layernorm(y, w, b), bl.layernorm(x, w, b)
    assert bool(out[4].isnan().all()) and torch.equal(out[keep], clean[keep])
    q, gamma, rs = bl.layernorm_quant_act(y, w, b)
    q0, gamma0, rs0 = bl.layernorm_quant_act(x, w, b)
    assert bool(gamma[4].isnan()) and bool(bl.dequant_act(q, gamma)[4].isnan().all())
    assert torch.equal(q[keep], q0[keep]) and torch.equal(gamma[keep], gamma0[keep]) and torch.equal(rs[keep], rs0[keep])


@pytest.mark.parametrize("N", [16, 203, 6912])
def test_checkpoint_keeps_nan(N):
    g, u = _rand(N, 5, N), _rand(N + 1, 5, N)
    g[2, N - 1] = float("nan")
    u[3, 0] = float("nan")
    c = bl.relu2_glu_quant_act(g, u)
    assert bool(c.gamma_g[2].isnan()) and bool(c.gamma_u[3].isnan())
    dg, du = bl.relu2_glu_backward(_rand(N + 2, 5, N), c.q_g, c.gamma_g, c.q_u, c.gamma_u)
    assert bool(dg[3].isnan().any()) and bool(torch.isfinite(dg[[0, 1, 4]].float()).all())
    assert bool(torch.isfinite(du[[0, 1, 4]].float()).all())


def test_norm_backward_nan_stays_in_its_row():
    M, K = 30, 2560
    x, dy = _rand(1, M, K), _rand(2, M, K)
    w = torch.rand(K, device=DEV)
    mean, rstd = _moments(x, 1e-5)
    dx, _, _ = bl.layernorm_backward(dy, x, w, mean, rstd)
    dy2 = dy.clone()
    dy2[7, 5] = float("nan")
    dx2, dw2, db2 = bl.layernorm_backward(dy2, x, w, mean, rstd)
    keep = [i for i in range(M) if i != 7]
    assert torch.equal(dx2[keep], dx[keep]) and bool(dx2[7].isnan().all())
    assert bool(dw2[5].isnan()) and int(dw2.isnan().sum()) == 1 and int(db2.isnan().sum()) == 1


def test_product_nan_stays_in_its_row():
    """A NaN in one row of dy reaches only that row of dx (few tokens and many) and, in one column, only that row of dW."""
    for M, N, K in [(20, 300, 200), (700, 300, 2048), (5000, 2560, 2560)]:
        w = bl.pack_ternary(torch.randint(-1, 2, (N, K), device=DEV, dtype=torch.int8, generator=_gen(1)), 0.02)
        dy = _rand(2, M, N)
        q, gamma = _checkpoint(3, M, K)
        dx, dW = bl.backward_input(w, dy), bl.backward_weight(dy, q, gamma)
        bad = dy.clone()
        bad[M // 3, 77] = float("nan")
        keep = [i for i in range(M) if i != M // 3]
        dx2 = bl.backward_input(w, bad)
        assert torch.equal(dx2[keep], dx[keep]) and bool(dx2[M // 3].isnan().all())
        dW2 = bl.backward_weight(bad, q, gamma)
        rows = [i for i in range(N) if i != 77]
        assert torch.equal(dW2[rows], dW[rows]) and bool(dW2[77].isnan().all())


# ---------------------------------------------------------------- widths and strides of every alignment
@pytest.mark.parametrize("K", [17, 31, 250, 2561, 2562, 2564, 5003, 12299])
@pytest.mark.parametrize("M", [1, 2, 150])
def test_every_alignment(M, K):
    """Rows that start anywhere in a 16-byte block, the first and the last of a buffer among them."""
    w, b = torch.rand(K, device=DEV) + 0.5, torch.rand(K, device=DEV)
    x, dy = _rand(M + K, M, K, outliers=True), _rand(M * K, M, K, scale=1e-3)
    mean, rstd = _moments(x, 1e-5)
    y, m1, r1 = bl.layernorm(x, w, b, 1e-5, want_stats=True)
    assert torch.equal(m1, mean) and torch.equal(r1, rstd) and torch.equal(y, _normed(x, w, b, mean, rstd).to(BF))
    q, gamma, rs = bl.layernorm_quant_act(x, w, b, 1e-5)
    q0, g0, rs0 = _codes(_normed(x, w, b, mean, rstd))
    assert torch.equal(q, q0) and torch.equal(gamma, g0) and torch.equal(rs, rs0)
    assert torch.equal(bl.dequant_act(q, gamma), _values(q, gamma).to(BF))
    dx, dw, db = bl.layernorm_backward(dy, x, w, mean, rstd)
    dx0, dw0, db0, size, dws, dbs = _norm_backward_ref(dy, x, w, mean, rstd, K)
    _close(dx, dx0, HALF * dx0.abs() * (1 + HALF) + 128 * U * size, "dx")
    _close(dw, dw0, (M + 200) * U * dws, "dw")
    c = bl.relu2_glu_quant_act(x, dy)
    for v, qq, gg in ((x, c.q_g, c.gamma_g), (dy, c.q_u, c.gamma_u), (_glu_h(x, dy), c.q_h, c.gamma_h)):
        q0, g0, _ = _codes(v.float())
        assert torch.equal(gg, g0) and torch.equal(qq, q0)
    dg, du = bl.relu2_glu_backward(dy, *c[:4])
    for off in range(1, 9, 3):  # the same values elsewhere in memory, rows apart and not
        for pad in (0, 5, 8):
            xs, ds = _strided(x, pad, off), _strided(dy, pad + 3, off)
            assert torch.equal(bl.layernorm(xs, w, b, 1e-5), y)
            for got, want in zip(bl.layernorm_quant_act(xs, w, b, 1e-5), (q, gamma, rs)):
                assert torch.equal(got, want)
            for got, want in zip(bl.layernorm_backward(ds, xs, w, mean, rstd), (dx, dw, db)):
                assert torch.equal(got, want)
            for got, want in zip(bl.relu2_glu_quant_act(xs, ds), c):
                assert torch.equal(got, want)
            for got, want in zip(bl.relu2_glu_backward(ds, *c[:4]), (dg, du)):
                assert torch.equal(got, want)
            assert torch.equal(bl.dequant_act(_strided(c.q_h, pad, off), c.gamma_h), bl.dequant_act(c.q_h, c.gamma_h))
