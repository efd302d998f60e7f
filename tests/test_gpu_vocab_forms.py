"""The vocabulary losses where one form of the computation meets the next: several
pieces of the vocabulary, the sizes at which single CTAs, CTA pairs and the kernel
for a few tokens take over, deep products, rows of very unequal magnitude."""

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


def _problem(T, V, D, dtype, seed=0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(T + V + D + seed)
    H = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
    W = (torch.randn(V, D, device="cuda", generator=gen) * spread / math.sqrt(D)).to(dtype)
    y = torch.randint(-1, V, (T,), device="cuda", generator=gen)
    return H, W, y, torch.randn(T, device="cuda", generator=gen) / T


def _run(h, H, W, y, dloss):
    loss, lse = h.xent(H, W, y)
    dH, dW = h.xent_grad(H, W, y, lse, dloss)
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


def _check(got, ref):
    for name, x in got.items():
        vr.check(name, x, ref[name])


def _reference(H, W, y, dloss):
    return vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(y, W.shape[0]), dloss, bf16=H.dtype == BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [100, 300, 700])
@pytest.mark.parametrize("piece", [256, 700, 1024])
def test_pieces_of_the_vocabulary(h, dtype, T, piece):
    """Any number of pieces gives the gradients, the last one shorter and not ending with a tile; both, or one alone."""
    V, D = 3001, 200
    H, W, y, dloss = _problem(T, V, D, dtype)
    h.set_option(sg.OPT_FORCE_VOCAB_PIECE, piece)
    got = _run(h, H, W, y, dloss)
    ref = _reference(H, W, y, dloss)
    _check(got, ref)
    dH, _ = h.xent_grad(H, W, y, got["lse"], dloss, need_dW=False)
    _, dW = h.xent_grad(H, W, y, got["lse"], dloss, need_dH=False)
    _check({"dH": dH, "dW": dW}, ref)


def test_piece_option_is_range_checked(h):
    for bad in (-1, 2 ** 31):
        with pytest.raises(sg.SgemmError):
            h.set_option(sg.OPT_FORCE_VOCAB_PIECE, bad)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2, 3, 4, 8, 9, 24, 25, 128, 129, 256, 257, 384, 385, 512, 513, 640, 641])
def test_token_counts_where_the_form_changes(h, dtype, T):
    H, W, y, dloss = _problem(T, 1500, 88, dtype)
    _check(_run(h, H, W, y, dloss), _reference(H, W, y, dloss))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [1024, 1025, 2100, 4097])
def test_deep_products(h, dtype, D):
    """Several accumulator segments, the last one short."""
    H, W, y, dloss = _problem(70, 600, D, dtype)
    _check(_run(h, H, W, y, dloss), _reference(H, W, y, dloss))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_tokens(h, dtype):
    """More tile rows than the kernels group."""
    H, W, y, dloss = _problem(4500, 300, 24, dtype)
    _check(_run(h, H, W, y, dloss), _reference(H, W, y, dloss))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [5, 200])
def test_rows_of_unequal_magnitude(h, dtype, T):
    """Rows of H and W from 1e-30 to 1e3 and rows of zeros: each is scaled by itself where FP32 is split."""
    V, D = 900, 64
    H, W, y, dloss = _problem(T, V, D, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    H = (H.float() * 10.0 ** torch.randint(-30, 3, (T, 1), device="cuda", generator=gen)).to(dtype)
    W = (W.float() * 10.0 ** torch.randint(-30, 1, (V, 1), device="cuda", generator=gen)).to(dtype)
    H[T // 2] = 0
    W[3], W[V - 1] = 0, 0
    _check(_run(h, H, W, y, dloss), _reference(H, W, y, dloss))


def test_a_head_of_zeros(h):
    """All logits equal: lse = log V, dH = 0."""
    T, V, D = 200, 700, 40
    H, _, y, dloss = _problem(T, V, D, F32)
    W = torch.zeros(V, D, device="cuda")
    got = _run(h, H, W, y, dloss)
    _check(got, _reference(H, W, y, dloss))
    assert (got["dH"] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2, 8])
def test_few_tokens_with_special_values(h, dtype, T):
    """The kernel for a few tokens: logits of thousands, and a token of NaN beside others."""
    V, D = 3000, 72
    H, W, y, dloss = _problem(T, V, D, dtype, spread=3000.0)
    y[:] = torch.arange(T, device="cuda")
    got = _run(h, H, W, y, dloss)
    ref = _reference(H, W, y, dloss)
    _check({k: got[k] for k in ("loss", "lse")}, ref)
    H = H.clone()
    H[1, 5] = math.nan
    loss, lse = h.xent(H, W, y)
    torch.cuda.synchronize()
    assert torch.isnan(loss[1]) and torch.isnan(lse[1])
    assert torch.equal(loss[0], got["loss"][0]) and torch.equal(lse[0], got["lse"][0])


@pytest.mark.parametrize("T", [3, 300])
def test_large_and_tiny_loss_gradients(h, T):
    """dloss from 1e-30 to 1e30 within a call, each token's row of dH to its own precision."""
    H, W, y, _ = _problem(T, 800, 48, F32)
    gen = torch.Generator(device="cuda").manual_seed(2)
    dloss = 10.0 ** torch.randint(-30, 31, (T,), device="cuda", generator=gen).float()
    _check(_run(h, H, W, y, dloss), _reference(H, W, y, dloss))
