"""The head-training command: the losses of its first step are the formulas', and training lowers them."""

import pytest

import dense_fp32_gemm_04_gb300 as sg
from dense_fp32_gemm_04_gb300 import head

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SIZES = dict(tokens=700, vocab=3001, width=120, features=64, entries=7)


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_first_step_is_gradient_descent_on_the_mixed_loss():
    """Loss and both weights after one step, against automatic differentiation in 64 bits.

    The products of this size leave at most about 1e-5 of a weight's change in FP32 (64 bits rounds nothing)."""
    T, V, D, F, n = (SIZES[k] for k in ("tokens", "vocab", "width", "features", "entries"))
    X, labels, ids, logits = head.make_data(torch, T, V, D, F, n)
    h = sg.Sgemm()
    s = head.Student(torch, h, V, D, F, torch.float32)
    P, W = (w.double().requires_grad_() for w in (s.P.clone(), s.W.clone()))
    tau, share, rate = 2.0, 0.3, 1.0
    got = s.step(X, X.T.contiguous(), labels, ids, logits, tau, share, rate)
    z = (X.double() @ P) @ W.T
    hard = torch.nn.functional.cross_entropy(z, labels, ignore_index=-100)
    used = labels >= 0
    q = torch.softmax(logits[used].double() / tau, 1)
    logp = torch.log_softmax(z[used] / tau, 1).gather(1, ids[used])
    soft = tau ** 2 * (q * (q.log() - logp)).sum(1).mean()
    loss = (1 - share) * hard + share * soft
    loss.backward()
    assert abs(got.item() - loss.item()) < 1e-5 * abs(loss.item())
    for w, ref in ((s.P, P), (s.W, W)):
        change = (w.double() - ref.detach()).norm()
        off = (w.double() - (ref.detach() - rate * ref.grad)).norm()
        # the weight itself is held in FP32: its rounding is beside what the products leave
        assert off < 1e-5 * change + 2.0 ** -24 * ref.norm()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    h.close()


@pytest.mark.parametrize("bf16", [False, True])
def test_training_lowers_the_loss(bf16):
    losses = head.train(torch, steps=30, bf16=bf16, **SIZES)
    assert losses[-1] < 0.7 * losses[0]
