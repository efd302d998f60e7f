"""The vocabulary losses at scales, logits, masks and strides where a number or an
argument leaves its range."""

import math

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import vocab_reference as vr  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_gemm_04_gb300 import _build

    _build.build()
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def _problem(T, V, D, dtype, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(T + V + D)
    H = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
    W = (torch.randn(V, D, device="cuda", generator=gen) * spread / math.sqrt(D)).to(dtype)
    return H, W, torch.randint(V, (T,), device="cuda", generator=gen), torch.randn(T, device="cuda", generator=gen) / T


def _check(h, got, ref):
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    for name, x in got.items():
        vr.check(name, x, ref[name])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1e-9, 1e-30, 1e-38])
@pytest.mark.parametrize("T", [3, 40, 300])
def test_scales_so_small_that_logits_vanish(h, T, scale, dtype):
    """Rows of zeros and of tiny numbers among others, a vocabulary that ends inside a tile: lse is log V."""
    V, D = 700, 72
    H, W, y, dloss = _problem(T, V, D, dtype)
    H[1] = 0.0
    H[2] = 1e-37
    loss, lse = h.xent(H, W, y, scale=scale)
    dH, dW = h.xent_grad(H, W, y, lse, dloss * (0.5 / scale), scale=scale)
    ref = vr.reference(H, W, scale, 1.0, *vr.xent_targets(y, V), dloss.double() * (0.5 / scale), bf16=dtype == BF16)
    _check(h, {"loss": loss, "lse": lse, "dH": dH, "dW": dW}, ref)


@pytest.mark.parametrize("temperature", [0.25, 0.5, 1.0, 3.0])
def test_teacher_logits_at_the_ends_of_their_type(h, temperature):
    """Logits that a division by the temperature would take out of FP32: only their differences count."""
    T, V, D, n = 40, 300, 32, 5
    H, W, _, dloss = _problem(T, V, D, F32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(V, (T, n), device="cuda", generator=gen)
    logits = torch.randn(T, n, device="cuda", generator=gen)
    far = torch.finfo(F32).max
    logits[0] = -far  # masked by the type's lowest value throughout: a uniform teacher
    logits[1, 1:] = -far  # one entry left
    logits[2] = far
    logits[3, :2], logits[3, 2:] = far, -far
    logits[4] = -math.inf  # masked
    logits[5, 1:] = -math.inf
    logits[6] = 2e38
    loss, lse = h.distill(H, W, ids, logits, temperature=temperature)
    dH, dW = h.distill_grad(H, W, ids, logits, lse, dloss, temperature=temperature)
    ref = vr.reference(H, W, 1 / temperature, temperature ** 2, *vr.teacher_targets(ids, logits, temperature, V), dloss)
    _check(h, {"loss": loss, "lse": lse, "dH": dH, "dW": dW}, ref)


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("masked", [1, 187, 600])
def test_the_mean_loss_after_a_masked_prompt(h, masked, op):
    """The first tokens are masked, as a prompt is, and dloss is one number for all.

    dZ held next to a power of two from below: off by at most 2^-7 / sqrt(12) / 1.98 = 1.1e-3 (2-norm), the result's
    rounding 1.6e-3, 2.0e-3 together; held anywhere, by up to 2^-8 for all tokens alike. 1 / 513 lies just below a power
    of two as well, so its rounding is the worst."""
    T, V, D = 513 + masked, 5000, 256
    H, W, y, _ = _problem(T, V, D, BF16, spread=0.5)
    y[:masked] = -100
    dloss = torch.full((T,), 1.0 / 513, device="cuda")
    if op == "xent":
        _, lse = h.xent(H, W, y)
        dH, dW = h.xent_grad(H, W, y, lse, dloss)
    else:
        ids, logits = torch.where(y < 0, -1, y)[:, None].contiguous(), torch.zeros(T, 1, device="cuda")
        _, lse = h.distill(H, W, ids, logits)
        dH, dW = h.distill_grad(H, W, ids, logits, lse, dloss)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(y, V), dloss, bf16=True)
    _check(h, {"dH": dH, "dW": dW}, ref)
    for name, got in (("dH", dH), ("dW", dW)):
        value = ref[name][0]
        off = ((got.cpu().double() - value).norm() / value.norm()).item()
        print(name, off)
        assert off < 2.3e-3, name


def test_row_strides_past_32_bits_are_refused(h):
    """The C entry points take strides as int: one that does not fit is an error, not its lower bits."""
    D = 8
    far = torch.empty(2 ** 32 + 2 * D, device="cuda", dtype=BF16).as_strided((2, D), (2 ** 32 + D, 1))
    near, y = torch.zeros(3, D, device="cuda", dtype=BF16), torch.zeros(3, device="cuda", dtype=torch.int64)
    lse = torch.zeros(3, device="cuda")
    with pytest.raises(ValueError, match="row stride"):
        h.xent(near, far, y)
    with pytest.raises(ValueError, match="row stride"):
        h.xent(far, near, y[:2])
    with pytest.raises(ValueError, match="row stride"):
        h.xent_grad(near[:2], near, y[:2], lse[:2], lse[:2], dH=far)
    with pytest.raises(ValueError, match="row stride"):
        h.xent_grad(near, near[:2], y, lse, lse, dW=far)
    del far
    torch.cuda.empty_cache()
