"""The vocabulary losses at the ends of what they promise about numbers: rows of W
of very unequal size, logits far past any model's, and what a masked token holds."""

import math

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import vocab_reference as vr  # noqa: E402

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


def _problem(T, V, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T + V + D)
    H = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
    W = (torch.randn(V, D, device="cuda", generator=gen) / math.sqrt(D)).to(dtype)
    return H, W, torch.randint(V, (T,), device="cuda", generator=gen), torch.randn(T, device="cuda", generator=gen) / T


def _finish(h):
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [math.nan, 1.7e-3, 0.0])
def test_what_dloss_of_a_masked_token_holds_changes_no_bit(h, dtype, value):
    """The first token's too, whose dloss sets how bfloat16 dZ is held."""
    H, W, y, dloss = _problem(300, 900, 72, dtype)
    y[0] = y[17] = -1
    _, lse = h.xent(H, W, y)
    want = h.xent_grad(H, W, y, lse, dloss)
    other = dloss.clone()
    other[0] = other[17] = value
    got = h.xent_grad(H, W, y, lse, other)
    _finish(h)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e8, 1e10])
def test_huge_logits_leave_gradients_within_the_probabilities_range(h, dtype, size):
    """lse is a multiple of 8 or 64 and more there, so p is only known to lie in [0, 1]: no gradient is larger than that gives."""
    T, V, D = 300, 900, 72
    H, W, y, dloss = _problem(T, V, D, dtype)
    H = (H.float() * size).to(dtype)
    _, lse = h.xent(H, W, y)
    dH, dW = h.xent_grad(H, W, y, lse, dloss)
    _finish(h)
    H, W, g = H.double(), W.double(), dloss.double().abs()
    # |dZ| <= |dloss|, 1 % for all roundings (bfloat16's are 2^-8 each)
    assert (dH.double().abs() <= 1.01 * g[:, None] * W.abs().sum(0)).all()
    assert (dW.double().abs() <= 1.01 * (g @ H.abs())).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2, 7, 20, 300])
@pytest.mark.parametrize("size", [1e8, 1e10, 1e30])
def test_huge_logits_leave_losses_to_their_precision(h, dtype, T, size):
    H, W, y, _ = _problem(T, 900, 72, dtype)
    H = (H.float() * size).to(dtype)
    loss, lse = h.xent(H, W, y)
    _finish(h)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(y, 900))
    vr.check("loss", loss, ref["loss"])
    vr.check("lse", lse, ref["lse"])


@pytest.mark.parametrize("large", [1e3, 1e6])
def test_one_row_of_the_head_far_larger_than_the_others(h, large):
    """FP32 dH: dZ is held to 2^-39 dloss times the largest |W| over its own row's largest."""
    T, V, D = 300, 900, 72
    H, W, y, dloss = _problem(T, V, D, F32)
    H[:, 0] = 0.0  # the large row's logit is 0
    W[7] = 0.0
    W[7, 0] = large
    _, lse = h.xent(H, W, y)
    dH, dW = h.xent_grad(H, W, y, lse, dloss)
    _finish(h)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(y, V), dloss)
    w = W.double().abs().cpu()
    held = 2.0 ** -39 * dloss.double().abs().cpu()[:, None] * (w.max() / w.amax(1))  # per entry of dZ
    vr.check("dH", dH, (ref["dH"][0], ref["dH"][1] + held @ w))
    vr.check("dW", dW, ref["dW"])
