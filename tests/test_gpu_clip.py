"""The global norm and clipping against their definition in 64 bits.

Tolerances: the norm is FP32 and sums lose at most 2^-21 of themselves (32 FP32 additions of squares, half of that in the
root), so 2^-20; outputs add the rounding of factor (two FP32 operations, 2^-23), of the product and of the type.
"""

import math

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import layers_reference as lr  # noqa: E402


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def make(shapes, seed, dtypes=(torch.float32, torch.bfloat16), scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(scale * torch.randn(s, device="cuda", generator=gen)).to(dtypes[i % len(dtypes)]) for i, s in enumerate(shapes)]


def check(norm, got, grads, max_norm):
    want, outs = lr.clip(grads, max_norm)
    assert norm.dtype == torch.float32 and norm.shape == ()
    assert abs(norm.item() - want) <= 2.0 ** -20 * want
    for a, b, g in zip(got, outs, grads):
        tol = 2.0 ** -20 + 2.0 ** -22 + torch.finfo(g.dtype).eps / 2
        assert ((a.double() - b).abs() <= tol * b.abs() + torch.finfo(g.dtype).smallest_normal).all()


SHAPES = {"one": [(1,)], "odd": [(3,), (1001,), (7, 13), (1, 5), (16383,), (16385,), (5, 20000), (33000, 2)],
          "some": [(64, 64)] * 31 + [(5,)], "many": [(i % 7 + 1, i + 1) for i in range(450)],
          "large": [(3001, 2047), (1 << 20,), (777,), (40, 50021)], "none": [(0,), (4, 0), (9,)]}


@pytest.mark.parametrize("name", sorted(SHAPES))
@pytest.mark.parametrize("share", [0.0, 0.3, 1.5, math.inf])
def test_against_64_bits(h, name, share):
    grads = make(SHAPES[name], len(name))
    keep = [g.clone() for g in grads]
    max_norm = share if math.isinf(share) else share * lr.clip(grads, 1.0)[0]
    outs = [torch.full_like(g, 7.0) for g in grads]
    norm = h.clip_grads(grads, max_norm, out=outs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    check(norm, outs, keep, max_norm)
    again = h.clip_grads(grads, max_norm)  # in place: the same bits
    torch.cuda.synchronize()
    assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))
    if share >= 1.5:
        assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


def test_rows_strides_and_alignment(h):
    """Views of larger buffers, what lies between their rows left alone; transposed and stepped ones."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    for dtype in (torch.float32, torch.bfloat16):
        base = torch.randn(50, 203, device="cuda", generator=gen).to(dtype)
        wide = torch.randn(3, 40000, device="cuda", generator=gen).to(dtype)
        line = torch.randn(1000, device="cuda", generator=gen).to(dtype)
        square = torch.randn(64, 96, device="cuda", generator=gen).to(dtype)
        views = lambda b, w, l, q: [b[:, 3:100], b[1:49, 101:], w[:, 8:39000], l[1:400], l[401::3], q.T]  # noqa: E731
        old = [t.clone() for t in (base, wide, line, square)]
        grads = views(base, wide, line, square)
        norm = h.clip_grads(grads, 0.5)
        torch.cuda.synchronize()
        check(norm, grads, views(*old), 0.5)
        touched = [torch.zeros_like(t, dtype=torch.bool) for t in old]
        for v in views(*touched):
            v.fill_(True)
        for t, o, m in zip((base, wide, line, square), old, touched):
            assert torch.equal(t[~m], o[~m])
        # outputs with strides of their own
        out = [torch.empty(50, 120, device="cuda", dtype=dtype)[:, 5:102], torch.empty(400, 2, device="cuda", dtype=dtype)[:399, 0]]
        norm = h.clip_grads([grads[0], grads[3]], 0.1, out=out)
        torch.cuda.synchronize()
        check(norm, out, [grads[0], grads[3]], 0.1)


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e-12, 1e12, 1e18, 3e19])
def test_norms_whose_squares_leave_fp32(h, scale):
    grads = make([(2000,), (33, 65), (8, 8)], 3, scale=scale)
    grads.append(torch.zeros(5000, device="cuda"))
    outs = [torch.empty_like(g) for g in grads]
    norm = h.clip_grads(grads, 0.01 * scale, out=outs)
    torch.cuda.synchronize()
    check(norm, outs, grads, 0.01 * scale)


def test_infinite_and_nan(h):
    for bad, value in ((math.inf, 0.0), (math.nan, math.nan)):
        grads = make([(100,), (3000,)], 4, dtypes=(torch.float32,))
        grads[1][777] = bad
        outs = [torch.empty_like(g) for g in grads]
        norm = h.clip_grads(grads, 1.0, out=outs)
        torch.cuda.synchronize()
        assert norm.isinf().item() if math.isinf(bad) else norm.isnan().item()
        rest = torch.cat([outs[0], outs[1][:777], outs[1][778:]])
        assert rest.isnan().all() if math.isnan(value) else (rest == 0).all()
        assert outs[1][777].isnan()
    norm = h.clip_grads([torch.full((3,), math.inf, device="cuda")], math.inf)
    assert norm.item() == math.inf


def test_no_tensors(h):
    assert h.clip_grads([], 1.0).item() == 0.0
    assert h.clip_grads([torch.empty(0, 5, device="cuda")], 1.0).item() == 0.0


def test_offsets_past_32_bits(h):
    """Elements beyond 2^32 bytes and 2^31 elements of one tensor count and are scaled."""
    n = (1 << 31) + 40001
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g[5], g[1 << 30], g[n - 1] = 3.0, 4.0, 12.0
    norm = h.clip_grads([g], 1.3)
    torch.cuda.synchronize()
    assert norm.item() == 13.0
    assert [g[i].item() for i in (5, 1 << 30, n - 1)] == [torch.tensor(x / 10).bfloat16().item() for x in (3.0, 4.0, 12.0)]
    assert g.count_nonzero().item() == 3


def test_graph_and_stream(h):
    grads = make([(100, 300), (5000,), (7,)] * 15, 8)
    outs = [torch.empty_like(g) for g in grads]
    h.reserve(sg.clip_workspace(len(grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = h.clip_grads(grads, 2.0, out=outs)
    for g in grads:
        g.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    check(norm, outs, grads, 2.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = h.clip_grads(grads, 2.0, stream=s)
    s.synchronize()
    assert torch.equal(second, norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_refusals(h):
    g = torch.ones(10, device="cuda")
    m = torch.ones(4, 6, 8, device="cuda")
    for err, call in (
            (TypeError, lambda: h.clip_grads([g.half()], 1.0)), (TypeError, lambda: h.clip_grads([1.0], 1.0)),
            (ValueError, lambda: h.clip_grads([g.cpu()], 1.0)), (ValueError, lambda: h.clip_grads([m[:, ::2, ::2]], 1.0)),
            (ValueError, lambda: h.clip_grads([g], 1.0, out=[])), (TypeError, lambda: h.clip_grads([g], 1.0, out=[g[:5]])),
            (TypeError, lambda: h.clip_grads([g], 1.0, out=[g.bfloat16()])), (ValueError, lambda: h.clip_grads([g[:1].expand(5)], 1.0)),
            (sg.SgemmError, lambda: h.clip_grads([g], -1.0)), (sg.SgemmError, lambda: h.clip_grads([g], math.nan)),
            (sg.SgemmError, lambda: h.clip_grads([g, g], 0.5))):
        with pytest.raises(err):
            call()
    torch.cuda.synchronize()
    assert (g == 1).all()


def test_tensors_over_each_other_are_refused(h):
    """Named twice, written over another tensor, or over its own with other rows: nothing is touched."""
    g, f, o = (torch.full((40, 6), x, device="cuda") for x in (1.0, 2.0, 3.0))
    for call in (lambda: h.clip_grads([g, g], 0.5, out=[o, f]), lambda: h.clip_grads([g, f], 0.5, out=[f, o]),
                 lambda: h.clip_grads([g, f], 0.5, out=[o, o]), lambda: h.clip_grads([g, f], 0.5, out=[f, g]),
                 lambda: h.clip_grads([g[:, :3]], 0.5, out=[g.view(-1)[:120].view(40, 3)])):
        with pytest.raises(sg.SgemmError):
            call()
    torch.cuda.synchronize()
    assert (g == 1).all() and (f == 2).all() and (o == 3).all()
    h.clip_grads([g, f], math.inf, out=[g, o])                       # its own tensor, and another one
    h.clip_grads([g[:, :3], g[:, 3:], f[:0], f[:0]], math.inf)       # neighbours, and tensors without elements
    torch.cuda.synchronize()
    assert (g == 1).all() and (f == 2).all() and (o == 2).all()
