"""Seeded random problems of the vocabulary losses (sizes, types, strides, offsets, pieces, math mode, masks, entries),
each output within the derived bounds; and calls of several handles at once."""

import math
import random

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import vocab_reference as vr  # noqa: E402


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_gemm_04_gb300 import _build

    _build.build()
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def _one(h, rng, gen):
    def log_uniform(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    T, V, D = log_uniform(1, 900), log_uniform(1, 4000), log_uniform(1, 1300)
    dtype = rng.choice([torch.bfloat16, torch.float32])
    pad, offset = rng.choice([0, 0, 1, 3, 8]), rng.choice([0, 0, 1, 8])
    tf32 = dtype == torch.float32 and rng.random() < 0.3

    def matrix(rows, cols, spread):
        flat = torch.zeros(offset + rows * (cols + pad), device="cuda", dtype=dtype)
        m = flat[offset:].view(rows, cols + pad)[:, :cols]
        return m.copy_(torch.randn(rows, cols, device="cuda", generator=gen) * spread)

    H, W = matrix(T, D, 1.0), matrix(V, D, rng.choice([0.5, 2.0]) / math.sqrt(D))
    dloss = torch.randn(T, device="cuda", generator=gen) * 10.0 ** rng.randint(-4, 3)
    h.set_math_mode(sg.MATH_TF32 if tf32 else sg.MATH_FP32)
    h.set_option(sg.OPT_FORCE_VOCAB_PIECE, rng.choice([0, 0, 256, 512, 1024]))
    if rng.random() < 0.5:
        labels, scale = torch.randint(-1, V + 1, (T,), device="cuda", generator=gen), rng.choice([1.0, 0.37, 3.0])
        loss, lse = h.xent(H, W, labels, scale=scale)
        dH, dW = h.xent_grad(H, W, labels, lse, dloss, scale=scale)
        targets, factor = vr.xent_targets(labels, V), 1.0
    else:
        n, tau = log_uniform(1, 200), rng.choice([1.0, 2.0, 0.5, 4.0])
        ids = torch.randint(-2, V + 1, (T, n), device="cuda", generator=gen)
        logits = torch.randn(T, n, device="cuda", generator=gen) * 5
        loss, lse = h.distill(H, W, ids, logits, temperature=tau)
        dH, dW = h.distill_grad(H, W, ids, logits, lse, dloss, temperature=tau)
        targets, scale, factor = vr.teacher_targets(ids, logits, tau, V), 1 / tau, tau * tau
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)
    ref = vr.reference(H, W, scale, factor, *targets, dloss, two_parts=tf32, bf16=dtype == torch.bfloat16)
    for name, x in (("loss", loss), ("lse", lse), ("dH", dH), ("dW", dW)):
        vr.check(f"{name} at {T} x {V} x {D}", x, ref[name])


@pytest.mark.parametrize("seed", range(8))
def test_random_problems(h, seed):
    rng, gen = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    for _ in range(50):
        _one(h, rng, gen)


def test_several_handles_at_once():
    """Three handles on three streams, their kernels in flight together, against their serial results, bit by bit."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator(device="cuda").manual_seed(0)
    jobs = []
    for T, dtype in ((700, torch.bfloat16), (300, torch.float32), (90, torch.bfloat16)):
        V, D = 6000, 512
        H = torch.randn(T, D, device="cuda", generator=gen).to(dtype)
        W = (torch.randn(V, D, device="cuda", generator=gen) / 16).to(dtype)
        labels = torch.randint(-1, V, (T,), device="cuda", generator=gen)
        jobs.append((sg.Sgemm(0), torch.cuda.Stream(), H, W, labels, torch.rand(T, device="cuda", generator=gen)))

    def run(job):
        handle, stream, H, W, labels, dloss = job
        loss, lse = handle.xent(H, W, labels, stream=stream)
        return (loss, lse) + handle.xent_grad(H, W, labels, lse, dloss, stream=stream)

    torch.cuda.synchronize()
    alone = []
    for job in jobs:
        alone.append(run(job))
        torch.cuda.synchronize()
    together = [[run(job) for job in jobs] for _ in range(10)]
    torch.cuda.synchronize()
    for round_ in together:
        for got, want in zip(round_, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    for job in jobs:
        assert job[0].check_device_status() == (sg.SGEMM_OK, 0)
        job[0].close()
