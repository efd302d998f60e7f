"""The vocabulary losses without a GPU: the 64-bit reference against differences,
planning, and what the entry points refuse before they touch anything."""

import ctypes
import itertools

import pytest

import dense_fp32_gemm_04_gb300 as sg

torch = pytest.importorskip("torch")

import vocab_reference as vr  # noqa: E402


@pytest.mark.parametrize("temperature", [1.0, 2.0])
def test_reference_gradients_against_differences(temperature):
    """The formula's gradients are the derivatives of the formula's losses (64 bits, central differences)."""
    gen = torch.Generator().manual_seed(3)
    T, V, D, n = 5, 23, 7, 4
    H, W = torch.randn(T, D, generator=gen).double(), torch.randn(V, D, generator=gen).double()
    ids = torch.randint(-1, V, (T, n), generator=gen)
    ids[2] = -1
    logits = torch.randn(T, n, generator=gen)
    targets = vr.teacher_targets(ids, logits, temperature, V)
    weights = torch.rand(T, generator=gen).double()

    def loss(a, b):
        return (vr.reference(a, b, 1 / temperature, temperature ** 2, *targets)["loss"][0] * weights).sum().item()

    ref = vr.reference(H, W, 1 / temperature, temperature ** 2, *targets, weights)
    e = 1e-5
    for which, grad in ((0, ref["dH"][0]), (1, ref["dW"][0])):
        way = torch.randn(grad.shape, generator=gen).double()
        up, down = [[H, W], [H, W]]
        up, down = list(up), list(down)
        up[which], down[which] = up[which] + e * way, down[which] - e * way
        assert abs((loss(*up) - loss(*down)) / (2 * e) - (grad * way).sum().item()) < 1e-7


@pytest.mark.parametrize("dtype,grad", list(itertools.product([sg.DTYPE_BF16, sg.DTYPE_F32], [False, True])))
def test_plan_covers_the_vocabulary(lib, dtype, grad):
    for T, V, D in [(1, 1, 1), (1, 131072, 4096), (60, 50021, 2048), (4096, 131072, 4096), (100000, 300000, 512),
                    (3000000, 1000, 64)]:
        for n in (0, 64):
            p = sg.vocab_plan(T, V, D, dtype=dtype, n=n, grad=grad)
            assert 1 <= p.piece <= V and (p.pieces - 1) * p.piece < V <= p.pieces * p.piece
            assert p.launches >= 1 and p.workspace_bytes > 0
            if not grad:
                assert p.pieces == 1
    # the logits' size is never in the workspace of a large gradient
    p = sg.vocab_plan(32768, 131072, 4096, dtype=dtype, grad=True)
    assert p.pieces > 1


def test_plan_copies_rows_off_their_lines(lib):
    """bfloat16 rows that are not 16-byte aligned are copied, from 2048 tokens on those off 128-byte lines too."""
    V, D = 50000, 1496

    def launches(T, align):
        return sg.vocab_plan(T, V, D, align_flags=align).launches

    for T in (500, 2047):
        assert launches(T, 0) == launches(T, 3) + 2 == launches(T, 15) + 2 == launches(T, 1) + 1
    for T in (2048, 9000):
        assert launches(T, 0) == launches(T, 3) == launches(T, 15) + 2 == launches(T, 7) + 1


def test_plan_refusals(lib):
    p = sg.VocabPlan()

    def plan(T=4, V=8, D=8, dtype=1, n=0, grad=0, align=3, sms=152, mode=0, out=ctypes.byref(p)):
        return lib.sgemm_vocab_plan(T, V, D, dtype, n, grad, align, sms, mode, out)

    assert plan() == sg.SGEMM_OK
    for bad in (dict(T=-1), dict(V=0), dict(D=0), dict(dtype=2), dict(dtype=-1), dict(n=-1), dict(grad=2),
                dict(align=16), dict(align=-1), dict(sms=0), dict(mode=5), dict(out=None)):
        assert plan(**bad) == sg.SGEMM_ERR_INVALID_VALUE, bad
    assert plan(n=1025) == sg.SGEMM_ERR_NOT_SUPPORTED


def test_null_handle_is_refused(lib):
    """Without a handle nothing is looked at, whatever the other arguments."""
    assert lib.sgemm_xent(None, 1, 4, 4, 1, None, 4, None, 4, None, 1.0, None, None, None) == sg.SGEMM_ERR_INVALID_VALUE
    assert lib.sgemm_xent_grad(None, 1, 4, 4, 1, None, 4, None, 4, None, 1.0, None, None, 0.0, None, 4, None, 4,
                               None) == sg.SGEMM_ERR_INVALID_VALUE
    assert lib.sgemm_distill(None, 1, 4, 4, 1, None, 4, None, 4, 2, None, None, 2, 1.0, None, None,
                             None) == sg.SGEMM_ERR_INVALID_VALUE
    assert lib.sgemm_distill_grad(None, 1, 4, 4, 1, None, 4, None, 4, 2, None, None, 2, 1.0, None, None, 0.0, None, 4,
                                  None, 4, None) == sg.SGEMM_ERR_INVALID_VALUE


def test_binding_refuses_what_is_not_a_device_matrix():
    """Type, device and shape errors are raised before the library is called (no GPU needed to see them)."""
    h = sg.Sgemm.__new__(sg.Sgemm)
    h.device, h._h, h._torch_device = 0, None, torch.device("cuda", 0)
    H, W = torch.zeros(3, 8), torch.zeros(5, 8)
    y = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        h.xent(H, W, y)  # host tensors
    with pytest.raises(TypeError):
        h.xent(H.double(), W.double(), y)
    with pytest.raises(TypeError):
        h.xent([[1.0]], W, y)
    with pytest.raises(TypeError):
        h.distill(H[0], W, y, y)
