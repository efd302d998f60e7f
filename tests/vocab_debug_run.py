"""Run by tests/test_gpu_vocab_debug.py in a process of its own, against the debug
build of the library (SGEMM_GB300_DEBUG_CHECKS=1): the vocabulary losses and their
gradients at small sizes of every form (single CTAs and pairs, few tokens, one and
several pieces, copied and split operands), the status word 0 after each."""

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import torch  # noqa: E402

import dense_fp32_gemm_04_gb300 as sg  # noqa: E402
import vocab_reference as vr  # noqa: E402

assert sg.LIB_PATH.endswith("_debug.so"), sg.LIB_PATH
h = sg.Sgemm(0)
calls = 0
gen = torch.Generator(device="cuda").manual_seed(0)
for dtype in (torch.bfloat16, torch.float32):
    for T, V, D, pad in ((1, 1, 1, 0), (2, 300, 64, 0), (5, 999, 130, 1), (20, 513, 72, 0), (100, 2000, 96, 0),
                         (129, 700, 65, 2), (300, 1025, 200, 0), (640, 300, 40, 8), (1100, 260, 513, 0)):
        W = torch.randn(V, D + pad, device="cuda", generator=gen).to(dtype)[:, :D] / D ** 0.5
        H = torch.randn(T, D + pad, device="cuda", generator=gen).to(dtype)[:, :D]
        g = torch.randn(T, device="cuda", generator=gen) / T
        y = torch.randint(-1, V, (T,), device="cuda", generator=gen)
        ids = torch.randint(-1, V, (T, 6), device="cuda", generator=gen)
        logits = torch.randn(T, 6, device="cuda", generator=gen)
        for targets, scale, factor, loss, grad in (
                (vr.xent_targets(y, V), 1.0, 1.0, lambda: h.xent(H, W, y), lambda s: h.xent_grad(H, W, y, s, g)),
                (vr.teacher_targets(ids, logits, 2.0, V), 0.5, 4.0, lambda: h.distill(H, W, ids, logits, temperature=2.0),
                 lambda s: h.distill_grad(H, W, ids, logits, s, g, temperature=2.0))):
            out, lse = loss()
            dH, dW = grad(lse)
            torch.cuda.synchronize()
            assert h.check_device_status() == (sg.SGEMM_OK, 0), (dtype, T, V, D)
            ref = vr.reference(H, W, scale, factor, *targets, g, bf16=dtype == torch.bfloat16)
            for name, x in (("loss", out), ("lse", lse), ("dH", dH), ("dW", dW)):
                vr.check(name, x, ref[name])
            calls += 2
h.close()
print(f"debug build: {calls} calls, status word 0 after each")
