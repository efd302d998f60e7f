"""Train a vocabulary head and the projection in front of it on labels and a teacher's top logits.

    python -m dense_fp32_gemm_04_gb300.head [--tokens 2048] [--vocab 32000] [--width 512] [--features 256]
                                            [--entries 16] [--temperature 2] [--share 0.5] [--steps 40] [--bf16]

A small student, ``logits = (X P) W^T``, learns from synthetic tokens: features X, the
labels that a hidden teacher of the same form draws, and the teacher's ``entries``
largest logits per token. Everything that costs anything runs in the library:

    H  = X P                       sgemm_run
    loss, lse                      sgemm_xent and sgemm_distill, mixed by ``share``
    dH, dW                         sgemm_xent_grad, then sgemm_distill_grad added to it (beta = 1)
    P  = P - rate * X^T dH         sgemm_run with alpha = -rate, beta = 1

The T x V logits exist nowhere. A tenth of the tokens are masked (label -100, no
teacher entries), as prompts are.
"""

from __future__ import annotations

import argparse

from . import Sgemm


def make_data(torch, tokens, vocab, width, features, entries, seed=0):
    """Features, labels and the teacher's best entries per token (ids -1 and label -100 where masked)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    X = rand(tokens, features)
    teacher = (X @ rand(features, width)) * (4.0 / (features * width) ** 0.5)
    head = rand(vocab, width)
    ids = torch.empty(tokens, entries, dtype=torch.int64, device="cuda")
    logits = torch.empty(tokens, entries, device="cuda")
    for r in range(0, tokens, 4096):  # the teacher's logits, some rows at a time
        top = (teacher[r:r + 4096] @ head.T).topk(entries, 1)
        ids[r:r + 4096], logits[r:r + 4096] = top.indices, top.values
    pick = torch.multinomial(torch.softmax(logits, 1), 1, generator=gen)
    labels = ids.gather(1, pick)[:, 0]
    masked = torch.rand(tokens, device="cuda", generator=gen) < 0.1
    labels[masked] = -100
    ids[masked] = -1
    return X, labels, ids, logits


class Student:
    """The student's weights, and one training step on them."""

    def __init__(self, torch, handle, vocab, width, features, dtype, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.torch, self.handle, self.dtype = torch, handle, dtype
        self.P = torch.randn(features, width, device="cuda", generator=gen) / features ** 0.5
        self.W = (torch.randn(vocab, width, device="cuda", generator=gen) * 0.05).to(dtype)

    def step(self, X, XT, labels, ids, logits, temperature, share, rate):
        """One step of gradient descent; the mean loss before it (a device tensor)."""
        torch, h = self.torch, self.handle
        T = X.shape[0]
        hidden = torch.empty(T, self.P.shape[1], device="cuda")
        h.run(X, self.P, hidden)
        H = hidden.to(self.dtype)
        hard, lse = h.xent(H, self.W, labels)
        soft, lse_soft = h.distill(H, self.W, ids, logits, temperature=temperature)
        used = (labels >= 0).sum()
        weight = (1.0 / used).expand(T).contiguous()
        dH, dW = h.xent_grad(H, self.W, labels, lse, weight * (1.0 - share))
        h.distill_grad(H, self.W, ids, logits, lse_soft, weight * share, temperature=temperature, dH=dH, dW=dW, beta=1.0)
        h.run(XT, dH.float(), self.P, alpha=-rate, beta=1.0)
        self.W.sub_(dW, alpha=rate)
        return ((1.0 - share) * hard + share * soft).sum() / used


def train(torch, tokens=2048, vocab=32000, width=512, features=256, entries=16, temperature=2.0, share=0.5, steps=40,
          rate=4.0, bf16=False):
    """Mean losses of `steps` steps on one batch."""
    X, labels, ids, logits = make_data(torch, tokens, vocab, width, features, entries)
    handle = Sgemm()
    student = Student(torch, handle, vocab, width, features, torch.bfloat16 if bf16 else torch.float32)
    XT = X.T.contiguous()
    losses = [student.step(X, XT, labels, ids, logits, temperature, share, rate) for _ in range(steps)]
    losses = torch.stack(losses).tolist()
    status, code = handle.check_device_status()
    handle.close()
    if status != 0:
        raise RuntimeError(f"device status {code:#x}")
    return losses


def main():
    import torch

    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, kind, default in (("tokens", int, 2048), ("vocab", int, 32000), ("width", int, 512), ("features", int, 256),
                                ("entries", int, 16), ("temperature", float, 2.0), ("share", float, 0.5), ("steps", int, 40),
                                ("rate", float, 4.0)):
        ap.add_argument("--" + name, type=kind, default=default)
    ap.add_argument("--bf16", action="store_true", help="hidden states and head in bfloat16")
    losses = train(torch, **vars(ap.parse_args()))
    for i, x in enumerate(losses):
        if i % 5 == 0 or i + 1 == len(losses):
            print(f"step {i:4d}  loss {x:.4f}")


if __name__ == "__main__":
    main()
