"""What the vocabulary losses refuse on a machine with a GPU: the arguments are
checked on the host, nothing is launched and no output is touched."""

import math

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T, V, D, N = 6, 40, 16, 3


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


@pytest.fixture
def x():
    f = dict(device="cuda", dtype=torch.float32)
    return {"H": torch.zeros(T, D, **f), "W": torch.zeros(V, D, **f), "y": torch.zeros(T, device="cuda", dtype=torch.int64),
            "ids": torch.zeros(T, N, device="cuda", dtype=torch.int64), "logits": torch.zeros(T, N, **f),
            "loss": torch.full((T,), 7.0, **f), "lse": torch.full((T,), 7.0, **f), "g": torch.zeros(T, **f),
            "dH": torch.full((T, D), 7.0, **f), "dW": torch.full((V, D), 7.0, **f)}


def test_c_entry_points(h, x):
    lib = sg.library()
    p = {k: t.data_ptr() for k, t in x.items()}

    def xent(T=T, V=V, D=D, dtype=0, H=p["H"], ldh=D, W=p["W"], ldw=D, y=p["y"], scale=1.0, loss=p["loss"], lse=p["lse"]):
        return lib.sgemm_xent(h.handle, T, V, D, dtype, H, ldh, W, ldw, y, scale, loss, lse, None)

    def distill(n=N, ids=p["ids"], logits=p["logits"], ldn=N, tau=1.0):
        return lib.sgemm_distill(h.handle, T, V, D, 0, p["H"], D, p["W"], D, n, ids, logits, ldn, tau, p["loss"],
                                 p["lse"], None)

    def grad(lse=p["lse"], dloss=p["g"], beta=0.0, dH=p["dH"], lddh=D, dW=p["dW"], lddw=D, scale=1.0):
        return lib.sgemm_xent_grad(h.handle, T, V, D, 0, p["H"], D, p["W"], D, p["y"], scale, lse, dloss, beta, dH,
                                   lddh, dW, lddw, None)

    bad = sg.SGEMM_ERR_INVALID_VALUE
    for case in (dict(T=-1), dict(V=0), dict(D=0), dict(dtype=3), dict(H=None), dict(W=None), dict(y=None),
                 dict(loss=None), dict(lse=None), dict(ldh=D - 1), dict(ldw=D - 1), dict(H=p["H"] + 2),
                 dict(W=p["W"] + 1), dict(y=p["y"] + 4), dict(loss=p["loss"] + 2), dict(scale=math.nan),
                 dict(scale=math.inf), dict(dtype=1, H=p["H"] + 1)):
        assert xent(**case) == bad, case
    for case in (dict(n=0), dict(n=-3), dict(ids=None), dict(logits=None), dict(ldn=N - 1), dict(tau=0.0),
                 dict(tau=-1.0), dict(tau=math.nan), dict(tau=math.inf), dict(ids=p["ids"] + 4),
                 dict(logits=p["logits"] + 2), dict(tau=1e-30), dict(tau=1e30)):
        assert distill(**case) == bad, case
    assert distill(n=1025, ldn=1025) == sg.SGEMM_ERR_NOT_SUPPORTED
    for case in (dict(lse=None), dict(dloss=None), dict(beta=math.nan), dict(lddh=D - 1), dict(lddw=D - 1),
                 dict(dH=p["dH"] + 2), dict(dW=p["dW"] + 1), dict(scale=math.nan)):
        assert grad(**case) == bad, case
    torch.cuda.synchronize()
    assert all((x[k] == 7).all() for k in ("loss", "lse", "dH", "dW"))
    assert xent() == distill() == sg.SGEMM_OK and grad() == sg.SGEMM_OK
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


def test_binding(h, x):
    H, W, y, ids, logits, lse, g = (x[k] for k in ("H", "W", "y", "ids", "logits", "lse", "g"))
    for err, call in (
            (TypeError, lambda: h.xent(H.bfloat16(), W, y)), (TypeError, lambda: h.xent(H, W, y.int())),
            (TypeError, lambda: h.xent(H.half(), W.half(), y)), (TypeError, lambda: h.xent(H.cpu(), W, y)),
            (ValueError, lambda: h.xent(H[:, :8], W, y)), (ValueError, lambda: h.xent(H, W, y[:3])),
            (ValueError, lambda: h.xent(H.T.contiguous().T, W, y)), (TypeError, lambda: h.xent(H, W, y.cpu())),
            (ValueError, lambda: h.distill(H, W, ids[:, :0], logits[:, :0])),
            (ValueError, lambda: h.distill(H, W, ids, logits[:, :2])),
            (TypeError, lambda: h.distill(H, W, ids, logits.double())),
            (ValueError, lambda: h.xent_grad(H, W, y, lse, g[:2])),
            (ValueError, lambda: h.xent_grad(H, W, y, lse, g, beta=1.0)),
            (TypeError, lambda: h.xent_grad(H, W, y, lse, g, dH=x["dH"].bfloat16())),
            (ValueError, lambda: h.xent_grad(H, W, y, lse, g, dW=x["dH"])),
            (ValueError, lambda: h.xent_grad(H, W, y, lse, g[:1].expand(T))),
            (sg.SgemmError, lambda: h.xent(H, W, y, scale=math.inf)),
            (sg.SgemmError, lambda: h.distill(H, W, ids, logits, temperature=0.0))):
        with pytest.raises(err):
            call()
