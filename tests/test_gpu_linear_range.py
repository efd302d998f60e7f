"""Linear layers over the whole range of their types: infinities, results next to FP32's ends, operands of very different sizes,
deep sums, and how exact FP32 results are.

Bounds for FP32 operands, per element of a product of a and b, mag = sum |a||b| over K: an operand is two float16 numbers, so it
is off by 2^-23 of itself, or by 2^-39 of the largest of its row (2^-25, half the last place of a float16 below 2^-14, where that
largest one lies in [2^14, 2^16)); the product of the two small parts, at most 2^-22 of |a||b|, is left out; sums of 256 products
are cut 16 times, by 4 * 2^-24 of what they have reached at most (the sums of the parts' other two products, 2^-11 of these, come
first), 2^-18 mag, and K / 256 of them are added in FP32. All together 2^-17 mag, K 2^-24 mag and 2^-38 (largest |a| of the row *
sum |b| + largest |b| * sum |a|). As a whole results are nearer, as sums grow from 0 and most cuts are smaller.
"""

import itertools
import math

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import layers_reference as lr  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
# few tokens, tiles split over clusters, whole tiles
FORMS = [(3, 300, 200), (150, 520, 200), (2200, 2400, 192)]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def rand(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def off(a, b, dtype):
    """What a product of the rows of a and b may be off by before it is rounded (infinities and NaN taken as 0)."""
    a, b = (x.double().nan_to_num(nan=0.0, posinf=0.0, neginf=0.0).abs() for x in (a, b))
    K, mag = a.shape[1], a @ b.T
    tol = mag * ((K + 32) * 2.0 ** -24 + 2.0 ** -17) + K * 2.0 ** -149  # (each sum is rounded to a multiple of 2^-149 at least)
    if dtype == F32:
        tol += 2.0 ** -38 * (a.max(1, keepdim=True).values * b.sum(1) + a.sum(1, keepdim=True) * b.max(1).values)
    return tol


def same(got, want, tol, dtype, partial=None):
    """Equal where want is infinite or NaN, else within tol and a rounding; results next to FP32's end may be on either side of it.
    partial: sum |a||b| of a form that adds unscaled products in FP32. Where that passes FP32's end, so may some of its products or
    sums, of either sign, and what comes after an infinity is no number that an FP32 sum in any order is held to."""
    most = torch.finfo(dtype).max
    got = got.double()
    half = torch.finfo(dtype).eps / 2
    near = (got - want).abs() <= tol + half * (want.abs() + tol) + 2.0 ** -149
    past = (want.abs() + tol >= most) & (got.isinf() | near) & ((got.sign() == want.sign()) | (want.abs() <= tol))
    inf = want.isinf() & (got == want)
    lost = ~got.isfinite() & (partial >= most) if partial is not None else False
    return bool((near | past | inf | (want.isnan() & got.isnan()) | lost).all())


def product(a, b):
    """The rows of a times those of b in 64 bits, with infinities and NaN as the formula has them whatever the library does."""
    clean = [x.double().nan_to_num(nan=0.0, posinf=0.0, neginf=0.0) for x in (a, b)]
    ref = clean[0] @ clean[1].T
    rows = (~a.isfinite()).any(1).nonzero()[:, 0].tolist()
    cols = (~b.isfinite()).any(1).nonzero()[:, 0].tolist()
    for r in rows:
        ref[r] = (a[r].double() * b.double()).sum(1)
    for c in cols:
        ref[:, c] = (a.double() * b[c].double()).sum(1)
    return ref


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_infinite_operands(h, M, N, K, dtype):
    """An infinity gives what the formula has: infinite results of its sign times the other operand's, NaN beside a zero."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    X, W, dY = rand(gen, M, K).to(dtype), rand(gen, N, K).to(dtype), rand(gen, M, N).to(dtype)
    X[1, 7], X[2, 9], W[5, 11], W[N - 1, K - 1] = math.inf, -math.inf, math.inf, -math.inf
    X[0, 11], W[17, 7] = math.inf, 0.0        # two infinities meet, and one meets a zero
    W[40, :] = torch.tensor(1.5).to(dtype)    # numbers that one part holds
    dY[1, 3], dY[M - 1, 6], dY[2, 17], X[2, 4] = math.inf, -math.inf, math.inf, 0.0
    Y = h.linear(X, W)
    dX, dW, _ = h.linear_grad(X, W, dY, need_db=False)
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    for got, a, b in ((Y, X, W), (dX, dY, W.T), (dW, dY.T, X.T)):
        want = product(a, b)
        assert want.isinf().any() and want.isnan().any()
        assert same(got, want, off(a, b, dtype), dtype)


# (X, W, dY) times these: results near both ends of FP32, though single operands and factors are far outside what they give
SCALES = [(1e33, 0.02, 1e-3), (1e35, 1.0, 1.0), (1e34, 1e-10, 1e-10), (1e-10, 1e34, 1e34), (1e-12, 1e-20, 1e36), (3e-39, 1e33, 1e30),
          (1e-20, 1e-17, 1e-20), (1e18, 1e18, 1e17), (1e30, 1e-39, 1e-3), (1e-44, 1e36, 1e-36)]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("M,N,K", FORMS + [(33, 2100, 2048), (40, 1, 1), (17, 4096, 1100), (16, 4096, 1100)])
def test_finite_results_are_finite(h, M, N, K, scale):
    """Both sides of the rule for few tokens (16 | 17 where W is large, 32 | 33 where it is small), split and whole tiles."""
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    X, W, dY = (rand(gen, *s) * f for s, f in zip(((M, K), (N, K), (M, N)), scale))
    b = rand(gen, N) * min(scale[0] * scale[1], 1e37)
    Y = h.linear(X, W, bias=b)
    dX, dW, _ = h.linear_grad(X, W, dY, need_db=False)
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    for name, got, a, c, add in (("Y", Y, X, W, b.double()), ("dX", dX, dY, W.T, 0.0), ("dW", dW, dY.T, X.T, 0.0)):
        ref = product(a, c)
        want = ref + add
        assert same(got, want, off(a, c, F32) + 2.0 ** -23 * want.abs(), F32), name


@pytest.mark.parametrize("M,N,K", FORMS + [(300, 600, 1030)])
def test_rows_and_columns_of_very_different_sizes(h, M, N, K):
    """Each row and each column of the operands has a size of its own, over most of FP32's range; dX's rows see the sizes of
    W's rows in its sum."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    sizes = lambda n, low, high: 10.0 ** (low + (high - low) * torch.rand(n, device="cuda", generator=gen))  # noqa: E731
    X = rand(gen, M, K) * sizes(M, -36, 36)[:, None]
    W = rand(gen, N, K) * sizes(N, -36, 36)[:, None]
    dY = rand(gen, M, N) * sizes(M, -30, 30)[:, None]
    Y = h.linear(X, W)
    dX, _, _ = h.linear_grad(X, W, dY, need_dW=False, need_db=False)
    torch.cuda.synchronize()
    few = X.double().abs() @ W.double().abs().T if sg.linear_plan(M, N, K, sg.DTYPE_F32).few else None
    assert same(Y, product(X, W), off(X, W, F32), F32, few)
    # W's sizes lie in dX's sum, so it is the products' sizes that count: every row of (dY times W's row sizes) has one largest
    size = W.double().abs().max(1).values
    assert same(dX, product(dY, W.T), off(dY.double() * size, (W.double() / size[:, None]).T, F32), F32)
    X = rand(gen, M, K) * sizes(K, -36, 36)
    dY = rand(gen, M, N) * sizes(N, -36, 36)
    _, dW, _ = h.linear_grad(X, W, dY, need_dX=False, need_db=False)
    torch.cuda.synchronize()
    assert same(dW, product(dY.T, X.T), off(dY.T, X.T, F32), F32)
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


@pytest.mark.parametrize("M,N,K", FORMS + [(130, 2301, 300)])
def test_zero_gradients_beside_large_weights(h, M, N, K):
    """Zeros of dZ (relu's slopes) stand where W's rows are large: dX is made of small rows alone, and is held as they are."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    W, dY = rand(gen, N, K), rand(gen, M, N)
    large = torch.rand(N, device="cuda", generator=gen) < 0.5
    large[0] = True
    W *= torch.where(large, 1e30, 1e-8)[:, None]
    dY *= 1e-20
    dY[:, large] = 0.0
    slope = (torch.rand(M, N, device="cuda", generator=gen) < 0.7).float()
    dX, _, _ = h.linear_grad(rand(gen, M, K), W, dY, slope, need_dW=False, need_db=False)
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    a, b = (dY * slope)[:, ~large], W[~large].T
    ref = product(a, b)
    assert (dX.double() - ref).norm() <= 5e-7 * ref.norm()
    assert same(dX, ref, off(a, b, F32), F32)


def test_deep_sums_of_one_sign(h):
    """bfloat16 sums of n products of one sign lose up to n 2^-27 of themselves: every 16 products are added to what the sum has
    reached, half of it on average, and it and they are cut to some 24 bits, together 4 * 2^-24 of it or less. What is near minus
    the result is added (as residual, as gradient so far), so that the rounding to bfloat16, 2^-8 of what is left, at most
    (2^-8 + n 2^-27) of the sum, hides none of that. (Means over results would say nothing: such sums differ by 1 / sqrt(n) of
    themselves, which is less than a step of bfloat16, so their roundings are alike.)"""
    gen = torch.Generator(device="cuda").manual_seed(12)
    uniform = lambda *s: (0.5 + torch.rand(*s, device="cuda", generator=gen)).to(BF16)  # noqa: E731

    def check(name, n, ref, call):
        near = -ref.to(BF16)
        left = call(near.clone())
        torch.cuda.synchronize()
        lost = n * 2.0 ** -27
        rounding = 2.0 ** -8 * (2.0 ** -8 + lost)
        far = (left.double() - (ref + near.double())) / ref
        assert -lost - rounding <= far.min().item() and far.max().item() <= rounding, (name, n, far.min().item(), far.max().item())

    for n in (4096, 65536, 300_007):
        X, dY, W = uniform(n, 200), uniform(n, 264), uniform(264, 200)
        check("dW", n, dY.double().T @ X.double(), lambda g: h.linear_grad(X, W, dY, dW=g, beta=1.0, need_dX=False, need_db=False)[1])
        A, B = uniform(150, n), uniform(136, n)
        check("Y", n, A.double() @ B.double().T, lambda g: h.linear(A, B, residual=g))
        G, V = uniform(150, n), uniform(n, 136)
        some = uniform(150, 136)
        check("dX", n, G.double() @ V.double(), lambda g: h.linear_grad(some, V, G, dX=g, beta=1.0, need_dW=False, need_db=False)[0])
        _, _, db = h.linear_grad(X, W, dY, need_dX=False, need_dW=False)
        ref = dY.double().sum(0)
        assert ((db.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -15) * ref).all()
    A, B = uniform(2600, 16384), uniform(2304, 16384)  # whole tiles
    check("Y", 16384, A.double() @ B.double().T, lambda g: h.linear(A, B, residual=g))
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


@pytest.mark.parametrize("M,N,K", FORMS + [(24, 2048, 4096), (300, 600, 8192), (2047, 3001, 1531), (64, 1000, 30000)])
def test_fp32_results_as_a_whole(h, M, N, K):
    """What the header says of FP32 results, in both math modes, which compute them alike."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    for sign in (False, True):
        X, W, dY = (rand(gen, *s) for s in ((M, K), (N, K), (M, N)))
        if sign:
            X, W, dY = X.abs(), W.abs(), dY.abs()
        most = 1.5e-6 if sign else 5e-7
        got = (h.linear(X, W),) + h.linear_grad(X, W, dY, need_db=False)[:2]
        h.set_math_mode(1)
        try:
            other = (h.linear(X, W),) + h.linear_grad(X, W, dY, need_db=False)[:2]
        finally:
            h.set_math_mode(0)
        torch.cuda.synchronize()
        for name, g, o, a, b in zip(("Y", "dX", "dW"), got, other, (X, dY, dY.T), (W, W.T, X.T)):
            assert torch.equal(g, o), name
            ref = product(a, b)
            assert (g.double() - ref).norm() <= most * ref.norm(), name
            assert same(g, ref, off(a, b, F32), F32), name
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


@pytest.mark.parametrize("M,N,K", FORMS[1:])
def test_small_elements_beside_large_ones(h, M, N, K):
    """One element of a row 2^e times the others, the other operand 0 in its place: the others are held to 2^-39 of it, so to
    2^(e - 39) of themselves, and are gone from e = 40 on. A few tokens lose nothing."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    for e in (10, 25, 32, 45):
        X, W, dY = ((1.0 + 0.5 * torch.rand(*s, device="cuda", generator=gen)) for s in ((M, K), (N, K), (M, N)))
        X[:, 3] *= 2.0 ** e
        W[:, 3] = 0.0
        dY[5] *= 2.0 ** e
        X0 = X.clone()
        X0[5] = 0.0
        few = h.linear(X[:3], W)
        Y = h.linear(X, W)
        dX, _, _ = h.linear_grad(X, W, dY, need_dW=False, need_db=False)
        _, dW, _ = h.linear_grad(X0, W, dY, need_dX=False, need_db=False)
        torch.cuda.synchronize()
        for name, got, a, b in (("Y", Y, X, W), ("dX", dX, dY, W.T), ("dW", dW, dY.T, X0.T)):
            assert same(got, product(a, b), off(a, b, F32), F32), (name, e)
        ref = product(X[:3], W)
        assert (few.double() - ref).norm() <= 5e-7 * ref.norm()
        if e >= 45:
            assert (Y == 0).all()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_bfloat16_activations_are_rounded_once(h, act):
    """Also where they are small: the tails are off by less than 2^-10.9 of themselves before they are rounded (2^-11 of the
    approximation; the exponent, up to 126, is rounded twice, by 2^-24 of itself, and 126 * 2^-23 log(2) is 2^-16.6). Down to
    z = -12.8, where the normal distribution's density is still above FP32's smallest normal number."""
    z = torch.cat([torch.linspace(-12.8, 12.8, 40001), -torch.logspace(-30, 1, 2000, base=2.0)]).cuda().to(BF16).unique()
    z = z[z >= -12.8][:, None].contiguous()
    one = torch.ones(1, 1, device="cuda", dtype=BF16)
    for rows in (z, *z.split(3)[::97]):
        Y = h.linear(rows, one, act=act)
        torch.cuda.synchronize()
        y, _ = lr.act(rows.double(), act)
        low = torch.finfo(F32).tiny * rows.double().abs().clamp_min(1)  # z times a factor that is flushed to 0 below 2^-126
        assert ((Y.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -10.9) * y.abs() + low).all(), act
