"""The vocabulary losses and their gradients on the GPU, against the formulas in
64 bits within derived bounds (vocab_reference.py), and against differences."""

import math

import pytest

import dense_fp32_gemm_04_gb300 as sg

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import vocab_reference as vr  # noqa: E402

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}

# (T, V, D): one of each, tile multiples and their neighbours, odd sizes, few and many
# of each, and vocabularies of several pieces
SIZES = [(1, 1, 1), (1, 2, 3), (2, 129, 8), (1, 5000, 64), (7, 300, 257), (16, 2050, 96), (17, 999, 130), (64, 256, 64),
         (65, 4099, 72), (127, 511, 65), (128, 512, 128), (129, 513, 127), (200, 33000, 40), (256, 1024, 256),
         (257, 777, 520), (500, 2000, 1100), (1030, 260, 33)]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_fp32_gemm_04_gb300 import _build

    _build.build()
    handle = sg.Sgemm(0)
    yield handle
    handle.close()


def _matrix(gen, rows, cols, dtype, pad=0, offset=0, spread=1.0):
    """rows x cols of normals at row stride cols + pad, `offset` elements into a buffer."""
    flat = torch.zeros(offset + rows * (cols + pad), device="cuda", dtype=TYPES[dtype])
    m = flat[offset:].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.randn(rows, cols, device="cuda", generator=gen) * spread)
    return m


def _operands(T, V, D, dtype, pad=0, offset=0, seed=0, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(1000 * T + 10 * V + D + seed)
    H = _matrix(gen, T, D, dtype, pad, offset)
    W = _matrix(gen, V, D, dtype, pad, offset, spread / math.sqrt(D))
    return H, W, gen


def _labels(gen, T, V, masked):
    y = torch.randint(V, (T,), device="cuda", generator=gen)
    return torch.where(torch.rand(T, device="cuda", generator=gen) < masked, -100, y)


def _entries(gen, T, V, n, short=True):
    ids = torch.randint(V, (T, n), device="cuda", generator=gen)  # duplicates are entries of their own
    logits = torch.randn(T, n, device="cuda", generator=gen) * 4
    if short:
        keep = torch.randint(0, n + 1, (T, 1), device="cuda", generator=gen)
        ids = torch.where(torch.arange(n, device="cuda") < keep, ids, -1)
    return ids, logits


def _status(h):
    torch.cuda.synchronize()
    assert h.check_device_status() == (sg.SGEMM_OK, 0)


def _check_all(h, got, ref):
    _status(h)
    for name, x in got.items():
        vr.check(name, x, ref[name])


def _xent(h, H, W, labels, dloss, scale=1.0, **more):
    loss, lse = h.xent(H, W, labels, scale=scale)
    dH, dW = h.xent_grad(H, W, labels, lse, dloss, scale=scale, **more)
    return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


def _distill(h, H, W, ids, logits, dloss, temperature=1.0, **more):
    loss, lse = h.distill(H, W, ids, logits, temperature=temperature)
    dH, dW = h.distill_grad(H, W, ids, logits, lse, dloss, temperature=temperature, **more)
    return {"loss": loss, "lse": lse, "dH": dH, "dW": dW}


def _dloss(gen, T):
    return torch.randn(T, device="cuda", generator=gen) / T


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES)
def test_xent(h, size, dtype):
    T, V, D = size
    H, W, gen = _operands(T, V, D, dtype)
    labels, dloss = _labels(gen, T, V, 0.2), _dloss(gen, T)
    got = _xent(h, H, W, labels, dloss, scale=0.75)
    _check_all(h, got, vr.reference(H, W, 0.75, 1.0, *vr.xent_targets(labels, V), dloss, bf16=dtype == BF16))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size,n,temperature", [((1, 1, 1), 1, 1.0), ((1, 3000, 64), 5, 2.0), ((33, 777, 65), 17, 0.5),
                                                ((129, 1025, 96), 64, 4.0), ((40, 2000, 48), 1024, 2.0),
                                                ((300, 513, 200), 100, 1.0), ((128, 33000, 40), 33, 2.0)])
def test_distill(h, size, n, temperature, dtype):
    T, V, D = size
    H, W, gen = _operands(T, V, D, dtype)
    ids, logits = _entries(gen, T, V, n)
    dloss = _dloss(gen, T)
    got = _distill(h, H, W, ids, logits, dloss, temperature)
    ref = vr.reference(H, W, 1 / temperature, temperature ** 2, *vr.teacher_targets(ids, logits, temperature, V), dloss,
                       bf16=dtype == BF16)
    _check_all(h, got, ref)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (3, 1), (0, 5), (16, 8)])
def test_strides_and_alignment(h, dtype, pad, offset):
    """Operands and results at row strides and offsets that are or are not 16-byte ones; nothing beside the results is written."""
    T, V, D = 130, 700, 136
    H, W, gen = _operands(T, V, D, dtype, pad, offset)
    labels, dloss = _labels(gen, T, V, 0.1), _dloss(gen, T)
    bufs = []
    for rows in (T, V):
        flat = torch.full((offset + rows * (D + pad) + 64,), 7.0, device="cuda", dtype=TYPES[dtype])
        bufs.append((flat, flat[offset:offset + rows * (D + pad)].view(rows, D + pad)))
    got = _xent(h, H, W, labels, dloss, dH=bufs[0][1][:, :D], dW=bufs[1][1][:, :D])
    _check_all(h, got, vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=dtype == BF16))
    for flat, m in bufs:
        assert (flat[:offset] == 7).all() and (flat[-64:] == 7).all() and (m[:, D:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_beta_adds_to_given_gradients(h, dtype):
    T, V, D = 200, 1500, 100
    H, W, gen = _operands(T, V, D, dtype)
    ids, logits = _entries(gen, T, V, 9)
    dloss = _dloss(gen, T)
    dH0, dW0 = _matrix(gen, T, D, dtype), _matrix(gen, V, D, dtype)
    got = _distill(h, H, W, ids, logits, dloss, 2.0, dH=dH0.clone(), dW=dW0.clone(), beta=-0.5)
    ref = vr.reference(H, W, 0.5, 4.0, *vr.teacher_targets(ids, logits, 2.0, V), dloss, bf16=dtype == BF16)
    u = 2.0 ** -8 if dtype == BF16 else 2 * vr.U
    for name, before in (("dH", dH0), ("dW", dW0)):
        value, bound = ref[name]
        value = value - 0.5 * before.cpu().double()
        ref[name] = (value, bound + u * value.abs() + vr.U * before.cpu().double().abs())
    _check_all(h, got, ref)


def test_one_gradient_alone(h):
    T, V, D = 150, 900, 64
    H, W, gen = _operands(T, V, D, BF16)
    labels, dloss = _labels(gen, T, V, 0.0), _dloss(gen, T)
    both = _xent(h, H, W, labels, dloss)
    dH, none = h.xent_grad(H, W, labels, both["lse"], dloss, need_dW=False)
    assert none is None
    none, dW = h.xent_grad(H, W, labels, both["lse"], dloss, need_dH=False)
    assert none is None
    assert h.xent_grad(H, W, labels, both["lse"], dloss, need_dH=False, need_dW=False) == (None, None)
    _status(h)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=True)
    vr.check("dH", dH, ref["dH"])
    vr.check("dW", dW, ref["dW"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masked_tokens(h, dtype):
    """Labels outside the vocabulary on either side mask; a masked token's dloss is not used, its gradient is exactly 0."""
    T, V, D = 140, 600, 64
    H, W, gen = _operands(T, V, D, dtype)
    labels = _labels(gen, T, V, 0.0)
    labels[3], labels[4], labels[5], labels[139], labels[70] = -1, V, 2 ** 40, -2 ** 63, V + 2 ** 32
    dloss = _dloss(gen, T)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=dtype == BF16)
    bad = dloss.clone()
    out = [3, 4, 5, 139, 70]
    bad[out] = math.nan
    got = _xent(h, H, W, labels, bad)
    _check_all(h, got, ref)
    assert (got["loss"][out] == 0).all() and (got["dH"][out] == 0).all()
    labels[:] = -100  # nothing left
    got = _xent(h, H, W, labels, bad)
    _status(h)
    assert (got["loss"] == 0).all() and (got["dH"] == 0).all() and (got["dW"] == 0).all()
    vr.check("lse", got["lse"], ref["lse"])


def test_teacher_entries_that_do_not_count(h):
    """Excluded entries may hold anything; -infinity is weight 0; empty and all -infinity lists mask; a NaN that counts shows."""
    T, V, D, n = 8, 400, 32, 6
    H, W, gen = _operands(T, V, D, F32)
    ids, logits = _entries(gen, T, V, n, short=False)
    ids[0, 1:4], logits[0, 1:4] = torch.tensor([-1, V, -2 ** 62], device="cuda"), torch.tensor(
        [math.nan, math.inf, -math.inf], device="cuda")
    logits[1, :5] = -math.inf
    ids[2] = -1
    logits[2] = math.nan
    logits[3] = -math.inf
    logits[4] = torch.finfo(torch.float32).min  # equal, far down: a softmax like any other
    ids[5] = 17  # one id six times
    dloss = _dloss(gen, T)
    got = _distill(h, H, W, ids, logits, dloss, 2.0)
    _check_all(h, got, vr.reference(H, W, 0.5, 4.0, *vr.teacher_targets(ids, logits, 2.0, V), dloss))
    for r in (2, 3):
        assert got["loss"][r] == 0 and (got["dH"][r] == 0).all()
    logits[6, 2] = math.nan
    loss, _ = h.distill(H, W, ids, logits, temperature=2.0)
    _status(h)
    assert torch.isnan(loss).tolist() == [r == 6 for r in range(T)]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_logits(h, dtype):
    """Logits of thousands: nothing overflows, the softmax is one entry or nearly so."""
    T, V, D = 70, 1300, 64
    H, W, gen = _operands(T, V, D, dtype, spread=3000.0)
    labels, dloss = _labels(gen, T, V, 0.1), _dloss(gen, T)
    got = _xent(h, H, W, labels, dloss)
    assert torch.isfinite(got["loss"]).all() and torch.isfinite(got["dH"].float()).all()
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=dtype == BF16)
    _check_all(h, {k: got[k] for k in ("loss", "lse")}, ref)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_not_a_number_stays_in_its_token(h, dtype):
    T, V, D = 300, 800, 48
    H, W, gen = _operands(T, V, D, dtype)
    labels = _labels(gen, T, V, 0.0)
    clean = h.xent(H, W, labels)
    H = H.clone()
    H[5, 7], H[258, 0] = math.nan, math.inf
    loss, lse = h.xent(H, W, labels)
    _status(h)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[5, 258]] = False
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
    assert not torch.isfinite(loss[5]) and not torch.isfinite(loss[258])


def test_two_parts_in_tf32_mode(h):
    T, V, D = 260, 1000, 300
    H, W, gen = _operands(T, V, D, F32)
    labels, dloss = _labels(gen, T, V, 0.1), _dloss(gen, T)
    h.set_math_mode(sg.MATH_TF32)
    try:
        got = _xent(h, H, W, labels, dloss)
    finally:
        h.set_math_mode(sg.MATH_FP32)
    _check_all(h, got, vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, two_parts=True))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bitwise_reproducible(h, dtype):
    T, V, D = 400, 5000, 260
    H, W, gen = _operands(T, V, D, dtype)
    ids, logits = _entries(gen, T, V, 12)
    dloss = _dloss(gen, T)
    a = _distill(h, H, W, ids, logits, dloss, 2.0)
    for _ in range(3):
        b = _distill(h, H, W, ids, logits, dloss, 2.0)
        assert all(torch.equal(a[k], b[k]) for k in a)
    _status(h)


def test_no_tokens(h):
    V, D = 300, 40
    H, W, gen = _operands(0, V, D, BF16)
    empty, dW0 = torch.empty(0, device="cuda"), _matrix(gen, V, D, BF16)
    labels = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = h.xent(H, W, labels)
    assert loss.shape == lse.shape == (0,)
    dH, dW = h.xent_grad(H, W, labels, empty, empty)
    _status(h)
    assert dH.shape == (0, D) and (dW == 0).all()
    dW = dW0.clone()
    h.xent_grad(H, W, labels, empty, empty, dH=dH, dW=dW, beta=0.5)
    _status(h)
    assert torch.equal(dW, (dW0.float() * 0.5).bfloat16())


@pytest.mark.parametrize("pad", [16328, 16327])
def test_offsets_beyond_32_bits(h, pad):
    """A head whose rows lie further than 2^31 elements apart from first to last, aligned and not."""
    T, V, D = 3, 140000, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    big = torch.zeros(V, D + pad, device="cuda", dtype=torch.bfloat16)
    W = big[:, :D]
    W.copy_(torch.randn(V, D, device="cuda", generator=gen) / 4)
    H = _matrix(gen, T, D, BF16)
    labels = torch.tensor([V - 1, V - 2, 0], device="cuda")
    dloss = _dloss(gen, T)
    loss, lse = h.xent(H, W, labels)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=True)
    _check_all(h, {"loss": loss, "lse": lse}, ref)
    out = torch.zeros(V, D + pad, device="cuda", dtype=torch.bfloat16)
    dH, dW = h.xent_grad(H, W, labels, lse, dloss, dH=torch.empty_like(H), dW=out[:, :D])
    _check_all(h, {"dH": dH, "dW": dW}, ref)
    assert (out[:, D:] == 0).all()
    del out, big
    torch.cuda.empty_cache()


def test_on_another_stream(h):
    """Inputs made on the side stream just before the call, outputs read on it just after: no synchronisation between."""
    T, V, D = 300, 9000, 256
    H, W, gen = _operands(T, V, D, BF16)
    labels, dloss = _labels(gen, T, V, 0.1), _dloss(gen, T)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        H2, W2 = H * 2, W * 0.5
        loss, lse = h.xent(H2, W2, labels)
        total = loss.sum()
    raw = h.xent(H2, W2, labels, stream=side)
    dH, dW = h.xent_grad(H2, W2, labels, raw[1], dloss, stream=side)
    side.synchronize()
    ref = vr.reference(H * 2, W * 0.5, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=True)
    _check_all(h, {"loss": loss, "lse": lse, "dH": dH, "dW": dW}, ref)
    assert torch.equal(raw[0], loss) and torch.isfinite(total)


def test_captured_into_a_graph():
    T, V, D, n = 200, 3000, 128, 7
    H, W, gen = _operands(T, V, D, BF16)
    ids, logits = _entries(gen, T, V, n)
    dloss = _dloss(gen, T)
    handle = sg.Sgemm(0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    small = sg.Sgemm(0)
    with pytest.raises(sg.SgemmError) as e:  # no workspace yet
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            small.distill(H, W, ids, logits, temperature=2.0)
    assert e.value.status == sg.SGEMM_ERR_NOT_SUPPORTED
    for grad in (False, True):
        handle.reserve(sg.vocab_plan(T, V, D, n=n, grad=grad).workspace_bytes)
    with torch.cuda.graph(graph, stream=side):
        got = _distill(handle, H, W, ids, logits, dloss, 2.0)
    H.copy_(_matrix(gen, T, D, BF16))
    graph.replay()
    ref = vr.reference(H, W, 0.5, 4.0, *vr.teacher_targets(ids, logits, 2.0, V), dloss, bf16=True)
    _check_all(handle, got, ref)
    small.close()
    handle.close()


@pytest.mark.parametrize("tokens", [1000, 700, 1023, 513])
def test_the_mean_loss_does_not_round_all_labels_alike(h, tokens):
    """dloss = 1 / tokens for all: the label's entry of dZ is that number times p - 1, p small for an untrained head.

    Where dZ is held next to a power of two from below, its rounding to 8 bits is at most 2^-7 / sqrt(12) / 1.98 = 1.1e-3
    of it (2-norm), the result's 2^-7 / sqrt(24) = 1.6e-3 for significands spread over [1, 2): 2.0e-3 together. Held
    anywhere it could be off by 2^-8 for all tokens alike."""
    V, D = 5000, 256
    H, W, gen = _operands(tokens, V, D, BF16, spread=0.5)
    labels = _labels(gen, tokens, V, 0.0)
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")
    got = _xent(h, H, W, labels, dloss)
    _status(h)
    ref = vr.reference(H, W, 1.0, 1.0, *vr.xent_targets(labels, V), dloss, bf16=True)
    for name in ("dH", "dW"):
        vr.check(name, got[name], ref[name])
        value = ref[name][0]
        assert (got[name].cpu().double() - value).norm() < 2.3e-3 * value.norm(), name


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_gradients_against_differences(h, op):
    """Directional derivatives of the summed loss by central differences of the library's own losses, FP32.

    The difference quotient at step e is off by at most e^2/6 |f'''| and by the losses' bounds over e; f''' of a
    log-sum-exp along a direction that moves a logit by at most m is at most 4 m^3 a token (third cumulant)."""
    T, V, D, n, tau = 40, 700, 96, 5, 2.0
    H, W, gen = _operands(T, V, D, F32)
    labels = _labels(gen, T, V, 0.1)
    ids, logits = _entries(gen, T, V, n)
    weights = torch.rand(T, device="cuda", generator=gen)
    if op == "xent":
        scale, factor, targets = 1.0, 1.0, vr.xent_targets(labels, V)
        loss = lambda a, b: h.xent(a, b, labels)[0]  # noqa: E731
        got = _xent(h, H, W, labels, weights)
    else:
        scale, factor, targets = 1 / tau, tau ** 2, vr.teacher_targets(ids, logits, tau, V)
        loss = lambda a, b: h.distill(a, b, ids, logits, temperature=tau)[0]  # noqa: E731
        got = _distill(h, H, W, ids, logits, weights, tau)
    dH, dW = got["dH"].double(), got["dW"].double()
    step = 2.0 ** -7
    for which in ("H", "W"):
        base = H if which == "H" else W
        way = torch.randn(base.shape, device="cuda", generator=gen).sign() * 2.0 ** -3
        lo, hi = base - step * way, base + step * way
        real = (hi.double() - lo.double()) / (2 * step)  # the direction as FP32 holds it
        a, b = (loss(hi, W), loss(lo, W)) if which == "H" else (loss(H, hi), loss(H, lo))
        w64 = weights.double()
        slope = ((a.double() - b.double()) * w64).sum().item() / (2 * step)
        want = ((dH if which == "H" else dW) * real).sum().item()
        move = scale * ((real @ W.double().T) if which == "H" else (H.double() @ real.T)).abs().amax(1)
        cubic = (factor * 4 * move ** 3 * w64).sum().item() * step ** 2 / 6
        ref = vr.reference(H, W, scale, factor, *targets, weights)
        noise = (2 * ref["loss"][1] * w64.cpu()).sum().item() / (2 * step)
        value, bound = ref["dH" if which == "H" else "dW"]
        grad = (bound.to("cuda") * real.abs()).sum().item()
        assert abs(slope - want) <= cubic + noise + grad, (which, slope, want, cubic, noise, grad)
        assert cubic + noise + grad < 0.2 * abs((value.to("cuda").abs() * real.abs()).sum().item())
    _status(h)
