"""How near the vocabulary losses come to 64 bits at deep products, as norms and as
signed means: what cutting the accumulation into segments is for.

The tensor core truncates its accumulator at each step of 16 products, by up to 2^-23 of
it and 2^-24 on average where it grows evenly from 0 (half of that, as it is half as large
on average, plus the alignment of the 16 products). s steps in a row lose at most s 2^-23
of a sum whose terms have one sign. So with one sign throughout
  a logit or lse  loses at most 64 steps: 2^-17 (bfloat16, 1024 deep), 32 and the parts'
                  small ones: 2^-18 (FP32, 512 deep); all of it toward zero. Undivided at
                  a width of 8192: 512 steps, 2^-14.
  FP32 dW         loses at most 16 steps of each segment, 2^-19, and the parts 2^-20; undivided
                  over 8192 tokens 2^-14.
The tests ask for half of the most that the segments can lose in a mean or a norm (the
average loss) and 2^-22 for the roundings beside it. An undivided sum loses eight times
that and more.
"""

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32
ROUNDINGS = 2.0 ** -22


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_gemm_04_gb300 import _build

    _build.build()
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def _status(h):
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


def _exact(H, W, y, dloss=None):
    a, b = H.double(), W.double()
    z = a @ b.T
    lse = torch.logsumexp(z, 1)
    out = {"lse": lse, "loss": lse - z.gather(1, y[:, None])[:, 0]}
    if dloss is not None:
        dz = (z - lse[:, None]).exp()
        dz[torch.arange(len(y)), y] -= 1.0
        dz *= dloss.double()[:, None]
        out.update(dH=dz @ b, dW=dz.T @ a)
    return out


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D", [(200, 2048), (200, 8192), (600, 4096)])
def test_lse_of_deep_products_of_one_sign(h, dtype, T, D):
    """All products of a logit positive, logits around 30: the signed mean error of lse, and that of the loss."""
    V = 1500
    gen = torch.Generator(device="cuda").manual_seed(D + T)
    H = (0.5 + torch.rand(T, D, device="cuda", generator=gen)).to(dtype)
    W = ((0.5 + torch.rand(V, D, device="cuda", generator=gen)) * (30.0 / D)).to(dtype)
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    loss, lse = h.xent(H, W, y)
    _status(h)
    want = _exact(H, W, y)
    most = 0.5 * (2.0 ** -17 if dtype == BF16 else 2.0 ** -18) + ROUNDINGS
    mean = ((lse.double() - want["lse"]).mean() / want["lse"].mean()).item()
    print("mean of lse", mean, "of", most)
    assert abs(mean) < most
    # the loss is a difference of two numbers that lose the same share: what is left is that of their difference
    size = want["lse"].abs().max().item()
    mean = (loss.double() - want["loss"]).mean().item()
    print("mean of loss", mean, "of", most * want["loss"].mean().item() + ROUNDINGS * size)
    assert abs(mean) < most * want["loss"].mean().item() + ROUNDINGS * size


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [2048, 4096])
def test_norms_of_a_training_step(h, dtype, D):
    """Hidden states that point at their labels, logits up to 30 of either sign."""
    T, V = 500, 3000
    gen = torch.Generator(device="cuda").manual_seed(D)
    W = (torch.randn(V, D, device="cuda", generator=gen) * 2 / D ** 0.5).to(dtype)
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    H = (torch.randn(T, D, device="cuda", generator=gen) + 4 * torch.rand(T, 1, device="cuda", generator=gen) * W[y].float()).to(dtype)
    dloss = (0.5 + torch.rand(T, device="cuda", generator=gen)) / T
    loss, lse = h.xent(H, W, y)
    dH, dW = h.xent_grad(H, W, y, lse, dloss)
    _status(h)
    want = _exact(H, W, y, dloss)
    most = 0.5 * (2.0 ** -17 if dtype == BF16 else 2.0 ** -18) + ROUNDINGS
    # errors of p are those of logits of up to 30 and the roundings of lse; bfloat16: dZ and the result rounded (uniform
    # over 2^-8 of a binade's end, 2^-7 / sqrt(12) at most each)
    grads = 30 * 2 * ROUNDINGS if dtype == F32 else 2.0 ** -7 / 6 ** 0.5
    for name, got, tolerance in (("loss", loss, most), ("lse", lse, most), ("dH", dH, grads), ("dW", dW, grads)):
        off = _off(got, want[name])
        print(name, off, "of", tolerance)
        assert off < tolerance, name


def test_deep_sums_of_one_sign_in_fp32_gradients(h):
    """dW sums over many tokens, all terms of one sign in the rows that are no token's label."""
    most = 0.5 * 2.0 ** -19 + 2.0 ** -20 + ROUNDINGS
    gen = torch.Generator(device="cuda").manual_seed(9)
    T, V, D = 8192, 300, 40
    H = 0.5 + torch.rand(T, D, device="cuda", generator=gen)
    W = (0.5 + torch.rand(V, D, device="cuda", generator=gen)) / D
    y = torch.randint(V, (T,), device="cuda", generator=gen) % 7
    dloss = (0.5 + torch.rand(T, device="cuda", generator=gen)) / T
    _, lse = h.xent(H, W, y)
    _, dW = h.xent_grad(H, W, y, lse, dloss)
    _status(h)
    off = _off(dW[7:], _exact(H, W, y, dloss)["dW"][7:])
    print((T, V, D), off, "of", most)
    assert off < most
