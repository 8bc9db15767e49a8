"""The gradient products' sums: exact where every partial sum is, and as precise as documented where they are not.

Integers.  dy of small whole numbers, codes with gamma = 127 (so that they are their own values, exact in bf16) or
ternary weights with a power of two for alpha: every partial sum is a whole number below 2^24, exact in fp32 in any
order, so that the results have to be equal: a slice of the reduction that is missing, doubled or misplaced shows.

Precision.  One step of the tensor cores adds 16 exact products to an fp32 sum and cuts the result off: less than one
last place, 2^-23, of the sum of magnitudes so far.  Over n steps with terms of one size these are i / n of the whole, so
n / 2 * 2^-23 of it in all.  A dW sum is cut into pieces of at most 56 steps (896 tokens), added up with one rounding
(2^-24) each; dx is one sum of N / 16 steps (every part of a split tile has fewer, and one rounding)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import ternary_weight_linear_fwd_b200 as bl  # noqa: E402
from test_gpu_training import BF, DEV, HALF, U, _close, _gen, _rand, _strided  # noqa: E402

STEP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ternary_weight_linear_fwd_b200 import build as b
    b.build()
    yield
    torch.cuda.synchronize()
    assert bl.device_status() == 0


def _restored(q, gamma):
    """x~ as defined, bf16 of RN32(q RN32(gamma / 127)): the quotient in 64 bits, rounded once (torch divides a CUDA
    tensor by a number as a product with its reciprocal, now and then the other neighbour, which one bf16 value in some
    ten thousand shows)."""
    scale = (gamma.double() / 127.0).float()
    return (q.float() * scale[:, None]).to(BF)


def _whole(seed, *shape, top=3):
    return torch.randint(-top, top + 1, shape, device=DEV, generator=_gen(seed)).to(BF)


# one sum and several pieces, expanded in place and restored, split and whole tiles, every remainder of a k-block
WEIGHT = [(1, 8, 16), (63, 65, 127), (64, 256, 256), (100, 203, 301), (777, 640, 2560), (832, 640, 640), (896, 512, 1024),
          (897, 640, 640), (1025, 257, 513), (2048, 640, 2560), (2048, 6912, 2560), (4096, 2600, 2100), (8000, 1300, 1500),
          (16384, 300, 520), (40000, 72, 136)]


@pytest.mark.parametrize("M,N,K", WEIGHT)
def test_weight_gradient_of_whole_numbers(M, N, K):
    dy = _whole(M + N, M, N)
    q = torch.randint(-127, 128, (M, K), device=DEV, generator=_gen(M + K), dtype=torch.int8)
    gamma = torch.full((M,), 127.0, device=DEV)
    want = (dy.double().t() @ q.double()).float()  # at most 40000 * 3 * 127 < 2^24
    dW = bl.backward_weight(dy, q, gamma)
    assert torch.equal(dW, want)
    assert torch.equal(bl.backward_weight(_strided(dy, 3, 1), _strided(q, 5, 3), gamma), want)
    out = dW.clone()
    bl.backward_weight(dy, q, gamma, out=out, accumulate=True)
    assert torch.equal(out, 2 * want)


# few tokens (one CTA and clusters), tiles expanded in place and restored, split and whole
INPUT = [(1, 20000, 8), (16, 2560, 6912), (17, 203, 301), (32, 2560, 2568), (33, 6912, 200), (70, 130, 264),
         (128, 2560, 6912), (257, 130, 1000), (700, 2563, 640), (777, 2560, 640), (2048, 6912, 2560), (4100, 8200, 2056),
         (300, 60000, 72)]


@pytest.mark.parametrize("M,N,K", INPUT)
@pytest.mark.parametrize("n,m", [(0, 0), (2, 4), (3, 8), (7, 8)])
def test_input_gradient_of_whole_numbers(M, N, K, n, m):
    if m and K % m:
        K = (K + m - 1) // m * m
    dy, add = _whole(M + N, M, N), _whole(M + K, M, K, top=100)
    if m:
        W = torch.randn(N, K, device=DEV, generator=_gen(n * m))
        w = bl.pack_weights(W, n, m)
        blocks = W.view(N, K // m, m)
        keep = torch.zeros_like(blocks).scatter_(2, blocks.abs().argsort(dim=2, descending=True, stable=True)[:, :, :n], 1)
        T = (torch.round(W / (w.alpha + 1e-5)).clamp(-1, 1) * keep.view(N, K)).to(torch.int8)
        w.alpha.fill_(0.25)
    else:
        T = torch.randint(-1, 2, (N, K), device=DEV, generator=_gen(N + K), dtype=torch.int8)
        w = bl.pack_ternary(T, 0.25)
    s = dy.double() @ T.double() * 0.25  # quarters, below 2^24 of them
    assert torch.equal(bl.backward_input(w, dy), s.to(BF))
    assert torch.equal(bl.backward_input(w, _strided(dy, 5, 1), add=add), (s + add.double()).to(BF))


# split tiles, and whole ones (74 of them) that a pair sums up alone: in one piece, in two, in eleven
@pytest.mark.parametrize("M,N,K", [(M, 264, 520) for M in (700, 896, 897, 1600, 2048, 8000, 16384)] +
                         [(M, 512, 9472) for M in (256, 512, 768, 832, 896, 960, 1536, 8192)])
@pytest.mark.parametrize("sign", [False, True])
def test_weight_gradient_precision(M, N, K, sign):
    """Independent of the number of tokens: the bound for terms of one sign, where every cut goes the same way, and the
    documented 1e-6 for terms of both."""
    dy = _rand(M, M, N, scale=1e-3)
    q = torch.randint(-127, 128, (M, K), device=DEV, generator=_gen(M + 1), dtype=torch.int8)
    gamma = 0.5 + torch.rand(M, device=DEV, generator=_gen(M + 2))
    if sign:
        dy, q = dy.abs(), q.abs()
    x = _restored(q, gamma).double()
    want, size = dy.double().t() @ x, dy.double().abs().t() @ x.abs()
    err = (bl.backward_weight(dy, q, gamma).double() - want).abs()
    # terms of random size: i / n of the whole to within a few percent after a handful of steps
    worst = (28 * 1.1 * STEP + (M // 768 + 2) * U)
    print(M, N, sign, "of the magnitudes", float((err / size).max()), "of the norm", float(err.norm() / want.norm()))
    _close(err, torch.zeros_like(err), worst * size, "dW")
    if not sign:
        assert float(err.norm() / want.norm()) < 1e-6


@pytest.mark.parametrize("M,N,K", [(16, 11008, 520), (300, 2560, 520), (300, 11008, 520), (300, 20000, 264),
                                   (2048, 6912, 640)])
@pytest.mark.parametrize("sign", [False, True])
def test_input_gradient_precision(M, N, K, sign):
    T = torch.randint(-1, 2, (N, K), device=DEV, generator=_gen(N), dtype=torch.int8)
    dy = _rand(M, M, N, scale=1e-3)
    if sign:
        T, dy = T.abs(), dy.abs()
    w = bl.pack_ternary(T, 0.037)
    alpha = float(w.alpha)
    want, size = dy.double() @ T.double() * alpha, dy.double().abs() @ T.double().abs() * alpha
    err = (bl.backward_input(w, dy).double() - want).abs()
    # the sum; the scale's rounding, a part's or warp's; one rounding to bf16
    cut = (N / 32 * 1.1 + 1) * STEP + 20 * U
    print(M, N, sign, float((err / size).max()), float(err.norm() / want.norm()))
    _close(err, torch.zeros_like(err), HALF * want.abs() * 1.01 + cut * size, "dx")
    assert float(err.norm() / want.norm()) < HALF
