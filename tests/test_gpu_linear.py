"""Linear layers and their gradients against the formulas in 64 bits.

Bounds, per element, u = 2^-24, mag = sum |a||b| over the product's K range:
  - accumulation: K u mag for FP32 additions in any order; the tensor cores truncate once per 16 products, which is less.
  - FP32 operands as three bfloat16 parts: the products left out are 2^-23 of |a||b| together, and 6 products of 256
    deep segments are 96 truncations of 2^-23 at most: 2^-16 mag. Two parts (TF32 mode): 3 * 2^-16 mag more.
  - a result is off by half a step of its type; dZ enters the products of bfloat16 operands rounded, 2^-8 of itself.
  - activations: 2^-20 of max(1, |z|) for the approximations, and 1.3 times what z is off by (no slope is above 1.13,
    no second derivative above 1.2); a slope held in 16 bits is off by 2^-15.
Integer operands whose sums stay below 2^24 are exact in every form; a result is then the exact sum rounded once.
"""

import itertools
import math
import random

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import layers_reference as lr  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


class Padded:
    """Rows in a larger buffer with canaries between and around them."""

    CANARY = -77.0

    def __init__(self, rows, cols, dtype, pad=0, offset=0, fill=None):
        self.buffer = torch.full((rows * (cols + pad) + offset + 64,), self.CANARY, device="cuda", dtype=dtype)
        self.m = self.buffer[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] if rows else \
            torch.empty(0, cols, device="cuda", dtype=dtype)
        if fill is not None:
            self.m.copy_(fill)

    def intact(self):
        other = torch.ones_like(self.buffer, dtype=torch.bool)
        if self.m.numel():
            other.as_strided(self.m.shape, self.m.stride(), self.m.storage_offset()).fill_(False)
        return bool((self.buffer[other] == self.CANARY).all())


def ints(gen, *shape, most=2):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=gen).float()


def rounded(x, dtype):
    return x.to(dtype).double()


def exact_case(h, M, N, K, dtype, pads=(0, 0, 0, 0), offset=0, act="none", bias=True, residual=True, beta=0.0, seed=0,
               need=(True, True, True)):
    """Integers: every form gives the exact sums, rounded once."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = Padded(M, K, dtype, pads[0], offset, ints(gen, M, K)).m
    W = Padded(N, K, dtype, pads[1], offset, ints(gen, N, K)).m
    b = Padded(1, N, dtype, 0, offset, ints(gen, 1, N)).m[0] if bias else None
    R = Padded(M, N, dtype, pads[2], offset, ints(gen, M, N)).m if residual else None
    out = Padded(M, N, dtype, pads[3], offset)
    Y, slope = h.linear(X, W, bias=b, act=act, residual=R, need_slope=True, out=out.m)
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    want, s = lr.linear(X, W, b, act, R)
    assert torch.equal(Y.double(), rounded(want.float(), dtype)), (M, N, K, dtype)
    assert out.intact()
    got = slope.double() * 2.0 ** -14 if dtype == BF16 else slope.double()
    assert torch.equal(got, s)
    dY = Padded(M, N, dtype, pads[2], offset, ints(gen, M, N)).m
    outs = [Padded(M, K, dtype, pads[3], offset, ints(gen, M, K)), Padded(N, K, dtype, pads[3], offset, ints(gen, N, K)),
            Padded(1, N, dtype, 0, offset, ints(gen, 1, N))]
    old = [o.m.double() for o in outs]
    dX, dW, db = h.linear_grad(X, W, dY, slope if act != "none" else None, dX=outs[0].m, dW=outs[1].m, db=outs[2].m[0],
                               beta=beta, need_dX=need[0], need_dW=need[1], need_db=need[2])
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    for given, got, ref, o, last in zip(need, (dX, dW, db), lr.linear_grad(X, W, dY, s), outs, old):
        assert (got is not None) == given
        expect = rounded((ref.view(last.shape) + beta * last).float(), dtype) if given else last
        assert torch.equal(o.m.double(), expect), (M, N, K, dtype)
        assert o.intact()


SIZES_M = (1, 2, 3, 4, 5, 8, 15, 16, 17, 24, 33, 64, 127, 128, 129, 255, 257, 300, 513)
SIZES_N = (1, 3, 7, 32, 63, 64, 65, 127, 128, 130, 255, 256, 257, 511, 1000)
SIZES_K = (1, 2, 7, 8, 9, 63, 64, 65, 128, 200, 255, 513, 1000)


@pytest.mark.parametrize("seed", range(60))
def test_integers_at_many_sizes(h, seed):
    rng = random.Random(seed)
    M, N, K = rng.choice(SIZES_M), rng.choice(SIZES_N), rng.choice(SIZES_K)
    dtype = rng.choice((BF16, F32))
    exact_case(h, M, N, K, dtype, pads=[rng.choice((0, 0, 1, 8)) for _ in range(4)], offset=rng.choice((0, 0, 1, 8)),
               act=rng.choice(("none", "relu")), bias=rng.random() < 0.7, residual=rng.random() < 0.6,
               beta=rng.choice((0.0, 1.0, -2.0)), seed=seed, need=rng.choice(list(itertools.product((True, False), repeat=3))[:7]))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K,form", [
    (1300, 2100, 130, "single or pairs"), (2500, 4000, 72, "pairs"), (2049, 2304, 200, "pairs"), (130, 20000, 96, "one row of tiles"),
    (20000, 200, 65, "one column"), (600, 1030, 2000, "split"), (257, 513, 5000, "split"), (64, 256, 9000, "split eight")])
def test_integers_in_every_form(h, M, N, K, form, dtype):
    for offset, pad, beta in ((0, 0, 0.0), (1, 3, 1.0)):
        exact_case(h, M, N, K, dtype, pads=(pad,) * 4, offset=offset, act="relu", beta=beta, seed=M + N)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_rows(h, dtype):
    exact_case(h, 0, 70, 33, dtype, beta=0.0)
    exact_case(h, 0, 70, 33, dtype, beta=2.0)


def real(M, N, K, dtype, seed, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    return ((spread * rand(M, K)).to(dtype), (rand(N, K) / K ** 0.5).to(dtype), (0.5 * rand(N)).to(dtype), rand(M, N).to(dtype),
            (rand(M, N) / M).to(dtype))


def product_bound(a, b, dtype, K, parts=3):
    """What a product of the rows of a and b may be off by before it is rounded."""
    mag = a.double().abs() @ b.double().abs().T
    return mag * ((K + 32) * 2.0 ** -24 + (0 if dtype == BF16 else 2.0 ** -16 + (3 * 2.0 ** -16 if parts == 2 else 0)))


@pytest.mark.parametrize("act", sorted(sg.ACTS))
@pytest.mark.parametrize("M,N,K,dtype,mode", [(3, 300, 200, BF16, 0), (3, 300, 200, F32, 0), (200, 700, 512, BF16, 0), (200, 700, 512, F32, 0),
                                              (200, 700, 512, F32, 1), (2200, 2400, 192, BF16, 0), (1400, 2400, 192, F32, 0)])
def test_against_64_bits(h, M, N, K, dtype, mode, act):
    X, W, b, R, dY = real(M, N, K, dtype, M + K, spread=2.0)
    h.set_math_mode(mode)
    try:
        Y, slope = h.linear(X, W, bias=b, act=act, residual=R, need_slope=True)
        dX, dW, db = h.linear_grad(X, W, dY, slope)
        plain = h.linear(X, W)
        torch.cuda.synchronize()
    finally:
        h.set_math_mode(0)
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    parts = 2 if mode == 1 else 3
    half = torch.finfo(dtype).eps / 2
    z = X.double() @ W.double().T + b.double()
    off = product_bound(X, W, dtype, K, parts) + 2.0 ** -23 * z.abs()
    y, s = lr.act(z, act)
    want = y + R.double()
    assert ((plain.double() - (z - b.double())).abs() <= off + half * (z - b.double()).abs() + 1e-30).all()
    tol = 1.3 * off + 2.0 ** -20 * z.abs().clamp_min(1) * (act != "none")
    assert ((Y.double() - want).abs() <= (tol + 2.0 ** -23 * want.abs()) + half * (want.abs() + tol)).all()
    got = slope.double() * 2.0 ** -14 if dtype == BF16 else slope.double()
    ok = (got - s).abs() <= tol + (2.0 ** -15 if dtype == BF16 else 2.0 ** -23)
    if act == "relu":
        ok |= z.abs() <= off
    assert ok.all()
    # gradients of the slopes that there are
    dz = dY.double() * got
    enters = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23
    for name, g, a, c, deep in (("dX", dX, dz, W.T, N), ("dW", dW, dz.T, X.T, M)):
        ref = a @ c.double().T
        tol = product_bound(a, c, dtype, deep, parts) + enters * (a.abs() @ c.double().abs().T)
        assert ((g.double() - ref).abs() <= tol + half * (ref.abs() + tol) + 1e-30).all(), name
    ref = dz.sum(0)
    tol = (M + 8) * 2.0 ** -24 * dz.abs().sum(0)
    assert ((db.double() - ref).abs() <= tol + half * (ref.abs() + tol)).all()
    if dtype == F32 and mode == 0:  # and as a whole: 96 truncations of half a step, of sums half as large on average, 2^-18.4
        for g, ref in ((plain, z - b.double()), (dX, dz @ W.double()), (dW, dz.T @ X.double())):
            assert (g.double() - ref).norm() <= 2.0 ** -18 * ref.norm()


def test_gradients_against_differences(h):
    """The layer's own change along a direction, in FP32, is what its gradients say."""
    M, N, K = 37, 90, 50
    for act in ("gelu", "gelu_tanh", "silu"):
        X, W, b, R, dY = real(M, N, K, F32, 5)
        _, slope = h.linear(X, W, bias=b, act=act, need_slope=True)
        dX, dW, db = h.linear_grad(X, W, dY, slope)
        e = 2.0 ** -7
        for t, g in ((X, dX), (W, dW), (b, db)):
            way = torch.randn(t.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
            at = []
            for sign in (e, -e):
                args = [u + sign * way if u is t else u for u in (X, W, b)]
                at.append((h.linear(args[0], args[1], bias=args[2], act=act).double() * dY.double()).sum())
            difference, said = ((at[0] - at[1]) / (2 * e)).item(), (g.double() * way.double()).sum().item()
            # the difference: e^2 of a third derivative, |z|' up to 8 here; and 2^-18 of the sums over 2 e
            scale = (dY.double().abs() * 8 ** 3 * e * e / 6).sum().item() * 0.2 + 2.0 ** -11 * dY.double().norm().item() * 10
            assert abs(difference - said) <= scale, (act, difference, said, scale)


def test_residual_in_place(h):
    for dtype, (M, N, K) in itertools.product((BF16, F32), ((3, 64, 96), (70, 300, 500), (2000, 2300, 130))):
        X, W, b, R, _ = real(M, N, K, dtype, 3)
        want = h.linear(X, W, bias=b, act="gelu", residual=R)
        got = h.linear(X, W, bias=b, act="gelu", residual=R, out=R)
        torch.cuda.synchronize()
        assert got is R and torch.equal(got, want)


def test_nan_and_infinity_stay_in_their_rows(h):
    for dtype, M in itertools.product((BF16, F32), (3, 150, 1500)):
        N, K = 2300, 100
        X, W, b, R, dY = real(M, N, K, dtype, 6)
        X[1, 5] = math.nan
        Y, slope = h.linear(X, W, bias=b, act="gelu", residual=R, need_slope=True)
        dX, _, _ = h.linear_grad(X, W, dY, slope, need_dW=False, need_db=False)
        torch.cuda.synchronize()
        keep = torch.arange(M, device="cuda") != 1
        for t in (Y, dX):
            assert t[1].isnan().all() and t[keep].isfinite().all()
        if dtype == BF16:
            assert (slope[1] == -32768).all()
        big = h.linear(torch.full_like(X, 3e18), torch.full_like(W, 3e18 if dtype == F32 else 3e18), act="none")
        torch.cuda.synchronize()
        assert (big.double() > 9e36 * K * 0.9).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_preactivations(h, dtype):
    """Every activation over the whole range of z, its slope with it: nothing but what the formula gives."""
    z = torch.cat([torch.linspace(-12, 12, 2001), torch.tensor([-3e4, -300.0, -50.0, 50.0, 300.0, 3e4, 1e15, -1e15, 1e25, -1e25])]).cuda()
    z = z.to(dtype)[:, None].contiguous()
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    for act in sorted(sg.ACTS):
        for rows in (z, z[:2]):
            Y, slope = h.linear(rows, one, act=act, need_slope=True)
            torch.cuda.synchronize()
            y, s = lr.act(rows.double(), act)
            s = s.nan_to_num(nan=0.0)
            got = slope.double() * 2.0 ** -14 if dtype == BF16 else slope.double()
            assert ((Y.double() - y).abs() <= 2.0 ** -20 * rows.double().abs().clamp_max(1e3) + torch.finfo(dtype).eps * y.abs()).all(), act
            far = rows.double().abs() > 1e3
            assert ((got - s).abs()[~far] <= 2.0 ** -14).all(), act
            assert ((got[far] == 0) | (got[far] == 1)).all() or act == "none"


def test_repeatable_and_on_other_streams(h):
    for dtype, (M, N, K) in itertools.product((BF16, F32), ((2, 500, 300), (300, 600, 700), (1500, 2500, 300))):
        X, W, b, R, dY = real(M, N, K, dtype, 4)
        first = h.linear(X, W, bias=b, act="silu", residual=R, need_slope=True)
        first += h.linear_grad(X, W, dY, first[1])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        second = h.linear(X, W, bias=b, act="silu", residual=R, need_slope=True, stream=s)
        second += h.linear_grad(X, W, dY, second[1], stream=s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, second))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(2, 300, 500), (200, 1000, 600), (1500, 2500, 300)])
def test_graphs(M, N, K, dtype):
    """A captured layer with its gradients, replayed on other values, from a handle that holds the plan's workspace."""
    h = sg.Sgemm(0)
    X, W, b, R, dY = real(M, N, K, dtype, 4)
    dt = sg.DTYPE_BF16 if dtype == BF16 else sg.DTYPE_F32
    align = 7 if N % 8 == 0 and K % 8 == 0 else 0
    h.reserve(max(sg.linear_plan(M, N, K, dt, grad, align).workspace_bytes for grad in (False, True)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, slope = h.linear(X, W, bias=b, act="gelu", residual=R, need_slope=True)
        dX, dW, db = h.linear_grad(X, W, dY, slope)
    for t, n in zip((X, W, b, R, dY), real(M, N, K, dtype, 44)):
        t.copy_(n)
    graph.replay()
    torch.cuda.synchronize()
    want = h.linear(X, W, bias=b, act="gelu", residual=R, need_slope=True)
    want += h.linear_grad(X, W, dY, want[1])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((Y, slope, dX, dW, db), want))
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    h.close()


def test_broadcast_and_shared_operands(h):
    """The same tensor as X and W, and as X and residual."""
    A = real(300, 300, 300, F32, 2)[0]
    Y = h.linear(A, A, residual=A)
    torch.cuda.synchronize()
    ref = A.double() @ A.double().T + A.double()
    assert (Y.double() - ref).norm() <= 2.0 ** -18 * ref.norm()


def test_refusals(h):
    X, W, b, R, dY = real(6, 40, 16, F32, 1)
    out = torch.full((6, 40), 7.0, device="cuda")
    slope = torch.ones(6, 40, device="cuda")
    for err, call in (
            (TypeError, lambda: h.linear(X.bfloat16(), W)), (TypeError, lambda: h.linear(X.half(), W.half())),
            (TypeError, lambda: h.linear(X.cpu(), W)), (TypeError, lambda: h.linear(X[0], W)), (ValueError, lambda: h.linear(X[:, :8], W)),
            (ValueError, lambda: h.linear(X, W, bias=b[:3])), (TypeError, lambda: h.linear(X, W, bias=b.bfloat16())),
            (ValueError, lambda: h.linear(X, W, act="tanh")), (ValueError, lambda: h.linear(X, W, residual=R[:, :8])),
            (ValueError, lambda: h.linear(X, W, out=out.T)), (TypeError, lambda: h.linear(X, W, out=out.bfloat16())),
            (ValueError, lambda: h.linear(X.T.contiguous().T, W)), (ValueError, lambda: h.linear(X, W, bias=torch.ones(80, device="cuda")[::2])),
            (ValueError, lambda: h.linear_grad(X, W, dY[:, :8])), (TypeError, lambda: h.linear_grad(X, W, dY, slope.bfloat16())),
            (TypeError, lambda: h.linear_grad(X, W, dY, slope.short())), (ValueError, lambda: h.linear_grad(X, W, dY, beta=1.0)),
            (ValueError, lambda: h.linear_grad(X, W, dY, dX=W)), (sg.SgemmError, lambda: h.linear_grad(X, W, dY, beta=math.inf, dX=X.clone(), dW=W.clone(), db=b.clone()))):
        with pytest.raises(err):
            call()
    lib, p = sg.library(), out.data_ptr()

    def layer(M=6, N=40, K=16, dtype=0, X=X.data_ptr(), ldx=16, W=W.data_ptr(), ldw=16, bias=None, act=0, R=None, ldr=0, Y=p, ldy=40,
              slope=None, lds=0):
        return lib.sgemm_linear(h.handle, M, N, K, dtype, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, slope, lds, None)

    def grad(M=6, slope=None, lds=0, dY=dY.data_ptr(), lddy=40, beta=0.0, dX=None, lddx=16, dW=None, lddw=16, db=None):
        return lib.sgemm_linear_grad(h.handle, M, 40, 16, 0, X.data_ptr(), 16, W.data_ptr(), 16, slope, lds, dY, lddy, beta, dX, lddx, dW,
                                     lddw, db, None)

    for case in (dict(M=-1), dict(N=0), dict(K=0), dict(dtype=2), dict(act=5), dict(act=-1), dict(X=None), dict(W=None), dict(Y=None),
                 dict(ldx=15), dict(ldw=15), dict(ldy=39), dict(R=p, ldr=39), dict(slope=p, lds=39), dict(X=p + 2), dict(bias=p + 1),
                 dict(Y=p + 2), dict(slope=p + 2, lds=40), dict(R=p + 3, ldr=40), dict(dtype=1, W=p + 1)):
        assert layer(**case) == sg.SGEMM_ERR_INVALID_VALUE, case
    for case in (dict(M=-1, dX=p), dict(dY=None, dX=p), dict(lddy=39, dX=p), dict(dX=p, lddx=15), dict(dW=p, lddw=15), dict(db=p + 2),
                 dict(beta=math.nan, dX=p), dict(slope=p, lds=39, dX=p)):
        assert grad(**case) == sg.SGEMM_ERR_INVALID_VALUE, case
    assert grad() == sg.SGEMM_OK  # nothing asked for
    torch.cuda.synchronize()
    assert (out == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [3, 48])
def test_outputs_over_operands_are_refused(h, M, dtype):
    """And nothing is touched; Y on the residual's own rows, and gradients over what the call does not read, are fine."""
    X, W, b, R, dY = real(M, 48, 48, dtype, 9)
    S = real(48, 48, 48, dtype, 10)[0]
    slope = h.linear(X, W, act="gelu", need_slope=True)[1]
    given = (X, W, b, R, dY, S)
    keep = [t.clone() for t in given]
    wide = torch.zeros(M, 96, device="cuda", dtype=dtype)
    for call in (lambda: h.linear(X, W, out=X), lambda: h.linear(S, W, residual=S, out=W), lambda: h.linear(X, S, residual=R, out=X),
                 lambda: h.linear(X, W, residual=wide[:, :48], out=wide.view(-1)[:M * 48].view(M, 48)),
                 lambda: h.linear_grad(X, W, dY, dX=dY), lambda: h.linear_grad(X, W, dY, dX=X), lambda: h.linear_grad(X, W, dY, dW=W),
                 lambda: h.linear_grad(S, W, S, dX=W, need_dW=False), lambda: h.linear_grad(S, S, dY=W, dX=S, dW=S)):
        with pytest.raises(sg.SgemmError):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(t, k) for t, k in zip(given, keep)) and (wide == 0).all()
    want = h.linear_grad(X, W, dY, slope)
    Y = h.linear(X, W, residual=R)
    assert h.linear(X, W, residual=R, out=R) is R
    h.linear_grad(X, W, dY, slope, dW=W, need_dX=False, need_db=False)   # W is not read for dW
    torch.cuda.synchronize()
    assert torch.equal(R, Y) and torch.equal(W, want[1])
    W.copy_(keep[1])
    h.linear_grad(X, W, dY, slope, dX=X, need_dW=False, need_db=False)   # nor X for dX
    torch.cuda.synchronize()
    assert torch.equal(X, want[0]) and h.check_device_status() == (sg.SGEMM_OK, 0)
