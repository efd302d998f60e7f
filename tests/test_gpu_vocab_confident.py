"""Gradients of tokens that the model is sure of: the label's entry of dZ is p - 1, so
the logits of the gradient call have to be those that its lse was made of.

Bounds: lse is stored in FP32, so p's relative error is at most e = 2^-22 (1 + |lse|) (its
own rounding, that of its factor ln 2 and the exponential, each 2^-24 of it or less). The
label's entry is off by e dloss, the others by e and what their logits lose to accumulation
and the label's does not, 1e-4, of themselves. dZ enters the products rounded to bfloat16
(2^-8) or in parts (2^-18 with all that the products of parts leave out), and a bfloat16
result is rounded once more. Every element of dH and dW is held to the sum of those. The inputs make 1 - p
about 1e-3 at a label's logit of 64: two calls that accumulate it differently (1e-6 to 4e-6
of it) miss by several times the bound.
"""

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_gemm_04_gb300 import _build

    _build.build()
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def _sure_tokens(T, V, D, dtype, pad=0, level=64.0, gap=14.0):
    """Token t has its label t at a logit of about `level`, all other entries about `gap` below."""
    gen = torch.Generator(device="cuda").manual_seed(T + V + D)
    half = D // 2

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float64)

    u, x = rand(half), rand(T, D - half)
    H = torch.empty(T, D + pad, device="cuda", dtype=dtype)[:, :D]
    W = torch.empty(V, D + pad, device="cuda", dtype=dtype)[:, :D]
    H.copy_(torch.cat([u.expand(T, half), x], 1))
    w = torch.cat([((level - gap) / u.square().sum() * u).expand(V, half), rand(V, D - half) * (0.02 / D ** 0.5)], 1)
    w[:T, half:] += gap * x / x.square().sum(1, keepdim=True)
    W.copy_(w)
    return H, W, torch.arange(T, device="cuda"), (0.5 + torch.rand(T, device="cuda", generator=gen)) / T


def _check(h, H, W, y, dloss, temperature=None):
    if temperature is None:
        scale, factor = 1.0, 1.0
        _, lse = h.xent(H, W, y)
        dH, dW = h.xent_grad(H, W, y, lse, dloss)
    else:
        scale, factor = 1 / temperature, temperature ** 2
        ids, logits = y[:, None].contiguous(), torch.zeros(len(y), 1, device="cuda")
        _, lse = h.distill(H, W, ids, logits, temperature=temperature)
        dH, dW = h.distill_grad(H, W, ids, logits, lse, dloss, temperature=temperature)
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    a, b = H.double(), W.double()
    logp = torch.log_softmax(scale * (a @ b.T), 1)
    p = logp.exp()
    rest = 1.0 - p.gather(1, y[:, None])[:, 0]
    rest = torch.where(rest > 1e-6, rest, 1e-6)
    assert 2e-4 < rest.min() and rest.max() < 5e-3  # the inputs are what they are meant to be
    g = factor * scale * dloss.double()[:, None]
    dz = g * p
    dz[torch.arange(len(y)), y] = -(g[:, 0] * rest)
    e = 2.0 ** -22 * (1 + lse.double().abs())[:, None]
    parts = 2.0 ** -8 if H.dtype == BF16 else 2.0 ** -18
    off = (e + 1e-4 + parts) * dz.abs()
    off[torch.arange(len(y)), y] += (g * e)[:, 0]
    for name, got, want, bound in (("dH", dH, dz @ b, off @ b.abs()), ("dW", dW, dz.T @ a, off.T @ a.abs())):
        bound = bound + parts * want.abs()
        worst = ((got.double() - want).abs() / bound).max().item()
        print(name, "worst", worst, "of the bound")
        assert worst <= 1.0, (name, worst)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [1024, 2048, 4096])
@pytest.mark.parametrize("T", [130, 500])
def test_sure_tokens(h, T, D, dtype):
    _check(h, *_sure_tokens(T, 1000, D, dtype))


@pytest.mark.parametrize("T,dtype,pad", [(1, BF16, 0), (2, BF16, 0), (8, BF16, 1), (1, F32, 0), (8, F32, 0), (24, F32, 3)])
@pytest.mark.parametrize("D", [1024, 4096])
def test_few_sure_tokens(h, T, D, dtype, pad):
    """Losses of a few tokens are accumulated in another way than their gradients' logits."""
    _check(h, *_sure_tokens(T, 1000, D, dtype, pad))


@pytest.mark.parametrize("T,dtype", [(200, BF16), (200, F32), (2, BF16), (20, F32)])
def test_sure_tokens_of_a_distillation(h, T, dtype):
    _check(h, *_sure_tokens(T, 1000, 4096, dtype, level=128.0, gap=28.0), temperature=2.0)
