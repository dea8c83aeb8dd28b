"""The RMS norm with a residual, its 8-bit form and its gradients against their formulas in 64 bits.

Bounds.  F is half a step of fp32, 2^-24, relative; u the output type's.  A sum of squares of N values adds at most
N / 64 of them one after another in a thread (a wave takes a row at the fewest), then at most 16 more; its terms
are positive, so it is off by (N / 64 + 16 + 3) F at most (3: the sum with the residual, twice, and the product).  The
factor r is its power -1/2, so half of that, and four roundings more (mean, eps, root, reciprocal); v has two products
and the rounding of the sum.  In all (N / 128 + 20) F relative: REL below, rounded up.
"""
import numpy as np
import pytest
import torch

import gemm_w4a16_amd as w
from test_gpu_memory_around_w8a8_experts import Arena

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
TYPES = {"bf16": (w.W4A16_BF16, torch.bfloat16, 2.0 ** -8, 0.0), "f16": (w.W4A16_FP16, torch.float16, 2.0 ** -11, 2.0 ** -25),
         "f32": (w.W4A16_FP32, torch.float32, F, 0.0)}
EPS = 1e-5


def REL(N):
    return (N / 128 + 24) * F


def data(T, N, kind, seed):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[kind][1]
    x, res = torch.randn((T, N), generator=g).to(dt), torch.randn((T, N), generator=g).to(dt)
    wt = (1 + 0.3 * torch.randn(N, generator=g)).to(dt)
    if T > 4:
        x[1], res[1] = 0, 0                    # nothing but eps
        x[2] = -res[2]                         # a sum of zeros
        x[3], res[3] = 0, 0
        x[3, N // 2] = 100.0                   # one value
    return x, res, wt


def reference(x, res, wt, eps=EPS):
    s = x.double() + (0 if res is None else res.double())
    v = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return s, v if wt is None else v * wt.double()


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 16), (37, 500), (6, 1001), (2000, 2048), (1030, 1000), (9, 8200), (2, 33333), (1, 40000),
          (1025, 64)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,N", SHAPES)
@pytest.mark.parametrize("with_res,with_w,with_h", [(1, 1, 1), (0, 1, 0), (1, 0, 0), (0, 0, 1)])
def test_norm(T, N, kind, with_res, with_w, with_h):
    act, dt, u, tiny = TYPES[kind]
    x, res, wt = data(T, N, kind, 3)
    res, wt = res if with_res else None, wt if with_w else None
    m = Arena()
    put = lambda t: None if t is None else m.put(t)
    h = m.out((T, N), dt) if with_h else None
    y = m.out((T, N), dt)
    w.w4a16_add_rmsnorm(act, put(x), put(res), T, N, put(wt), EPS, h, y)
    s, v = reference(x, res, wt)
    if with_h:
        assert torch.equal(h.cpu(), (x.float() + (0 if res is None else res.float())).to(dt))
    err = (y.cpu().double() - v).abs() - ((u + (1 + u) * REL(N)) * v.abs() + tiny)
    assert err.max().item() <= 0
    m.check()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,N", [(1, 16), (1, 4096), (3, 48), (37, 2080), (2000, 2048), (1030, 1008), (9, 8208), (2, 33328)])
@pytest.mark.parametrize("with_res,with_w", [(1, 1), (0, 0)])
def test_norm_i8(T, N, kind, with_res, with_w):
    act, dt, _, _ = TYPES[kind]
    x, res, wt = data(T, N, kind, 5)
    res, wt = res if with_res else None, wt if with_w else None
    m = Arena()
    put = lambda t: None if t is None else m.put(t)
    dx, dres, dw = put(x), put(res), put(wt)
    h, xq, a = m.out((T, N), dt), m.out((T, N), torch.int8), m.out((T,), torch.float32)
    w.w4a16_add_rmsnorm_i8(act, dx, dres, T, N, dw, EPS, h, xq, a)
    assert torch.equal(h.cpu(), (x.float() + (0 if res is None else res.float())).to(dt))
    _, v = reference(x, res, wt)
    top = v.abs().amax(1)
    ref = torch.where(top == 0, torch.ones_like(top), top / 127)
    a64 = a.cpu().double()
    assert ((a64 - ref).abs() <= (REL(N) + 2 * F) * ref).all()
    # a code is at most half a step from v / a as divided in fp32 (one rounding), v is off by REL
    err = (xq.cpu().double() * a64[:, None] - v).abs()
    assert (err <= a64[:, None] * (0.5 + 128 * 2 * F) + REL(N) * v.abs()).all()
    assert (xq.cpu().abs().amax(1) == torch.where(top == 0, 0, 127)).all()
    m.check()
    if kind == "f32":  # of fp32 rows: the codes of the norm's own output, bit for bit
        y, xq2, a2 = m.out((T, N), dt), m.out((T, N), torch.int8), m.out((T,), torch.float32)
        w.w4a16_add_rmsnorm(act, dx, dres, T, N, dw, EPS, None, y)
        w.w4a16_quantize_rows_i8(act, y, T, N, xq2, a2)
        assert torch.equal(xq, xq2) and torch.equal(a, a2)


def test_codes_next_to_a_border():
    """Values on and next to the borders between codes, which a product with the scale's reciprocal would miss: rows of
    magnitude one, so that the norm leaves them as they are, up to its factor."""
    N, T = 256, 64
    q = torch.arange(N, dtype=torch.float64) % 127 + 0.5
    x = torch.zeros((T, N))
    for t in range(T):
        for i in range(N):
            x[t, i] = float(np.float32(q[i] / 127 * (1 + (t - 32) * 2.0 ** -24)))
    x[:, 0] = 1.0
    xq, a = torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y, xq2, a2 = torch.empty((T, N), device="cuda"), torch.empty_like(xq), torch.empty_like(a)
    w.w4a16_add_rmsnorm_i8(w.W4A16_FP32, x.cuda(), None, T, N, None, 0.0, None, xq, a)
    w.w4a16_add_rmsnorm(w.W4A16_FP32, x.cuda(), None, T, N, None, 0.0, None, y)
    yn = y.cpu().numpy()
    an = np.abs(yn).max(1) / np.float32(127)
    np.testing.assert_array_equal(a.cpu().numpy(), an)
    np.testing.assert_array_equal(xq.cpu().numpy(), np.clip(np.rint(yn / an[:, None]), -127, 127).astype(np.int8))


def test_codes_next_to_a_border_with_a_small_eps():
    """The same rows with an eps that is lost beside their mean square, which other kernels take than eps = 0: as many of the
    values lie on borders."""
    N, T, eps = 256, 64, 2.0 ** -60
    q = np.arange(N) % 127 + 0.5
    x = np.stack([(q / 127 * (1 + (t - 32) * 2.0 ** -24)).astype(np.float32) for t in range(T)])
    x[:, 0] = 1.0
    x = torch.from_numpy(x).cuda()
    xq, a, y = torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.empty((T, N), device="cuda")
    w.w4a16_add_rmsnorm_i8(w.W4A16_FP32, x, None, T, N, None, eps, None, xq, a)
    w.w4a16_add_rmsnorm(w.W4A16_FP32, x, None, T, N, None, eps, None, y)
    yn = y.cpu().numpy()
    an = np.abs(yn).max(1) / np.float32(127)
    np.testing.assert_array_equal(a.cpu().numpy(), an)
    np.testing.assert_array_equal(xq.cpu().numpy(), np.clip(np.rint(yn / an[:, None]), -127, 127).astype(np.int8))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("N", [512, 1001, 9000])
def test_in_place(kind, N):
    """h in residual's own array and y in x's, in whole units and not, with rows longer than a block holds."""
    act, dt, _, _ = TYPES[kind]
    T = 7
    x, res, wt = (t.cuda() for t in data(T, N, kind, 7))
    h, y = torch.empty_like(x), torch.empty_like(x)
    w.w4a16_add_rmsnorm(act, x, res, T, N, wt, EPS, h, y)
    x2, r2 = x.clone(), res.clone()
    w.w4a16_add_rmsnorm(act, x2, r2, T, N, wt, EPS, r2, x2)
    assert torch.equal(r2, h) and torch.equal(x2, y)
    x2, r2 = x.clone(), res.clone()
    w.w4a16_add_rmsnorm(act, x2, r2, T, N, wt, EPS, x2, r2)
    assert torch.equal(x2, h) and torch.equal(r2, y)
    if N % 16 == 0:
        xq, a = torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        xq2, a2 = torch.empty_like(xq), torch.empty_like(a)
        w.w4a16_add_rmsnorm_i8(act, x, res, T, N, wt, EPS, None, xq, a)
        r2 = res.clone()
        w.w4a16_add_rmsnorm_i8(act, x, r2, T, N, wt, EPS, r2, xq2, a2)
        assert torch.equal(xq, xq2) and torch.equal(a, a2) and torch.equal(r2, h)


# rows in turn, the next asked for before one is written
@pytest.mark.parametrize("kind,T,N", [("bf16", 9000, 512), ("f32", 700, 16000), ("f16", 1100, 4001), ("bf16", 300, 40000)])
def test_many_rows_in_place(kind, T, N):
    act = TYPES[kind][0]
    x, res, wt = (t.cuda() for t in data(T, N, kind, 17))
    h, y = torch.empty_like(x), torch.empty_like(x)
    w.w4a16_add_rmsnorm(act, x, res, T, N, wt, EPS, h, y)
    x2, r2 = x.clone(), res.clone()
    w.w4a16_add_rmsnorm(act, x2, r2, T, N, wt, EPS, r2, x2)
    assert torch.equal(r2, h) and torch.equal(x2, y)
    dy, dh = torch.randn_like(x), torch.randn_like(x)
    ws, nb = w.alloc_add_rmsnorm_backward_workspace(T, N)
    dx, dw, dw2 = torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    w.w4a16_add_rmsnorm_backward(act, dy, dh, h, T, N, wt, EPS, dx, dw, ws, nb)
    w.w4a16_add_rmsnorm_backward(act, dy, dh, h, T, N, wt, EPS, dh, dw2, ws, nb)
    assert torch.equal(dx, dh) and torch.equal(dw, dw2)


def test_longest_rows():
    """Of 2^22 elements, the most that a call takes."""
    T, N = 3, 1 << 22
    test_norm(T, N, "bf16", 1, 1, 1)
    test_norm_i8(T, N, "f16", 1, 1)
    test_gradients(T, N, "bf16", 1, 1)


def test_in_place_long_i8():
    T, N = 3, 16 * 1600
    x, res, wt = (t.cuda() for t in data(T, N, "bf16", 8))
    xq, a, h = torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
    xq2, a2, x2 = torch.empty_like(xq), torch.empty_like(a), x.clone()
    w.w4a16_add_rmsnorm_i8(w.W4A16_BF16, x, res, T, N, wt, EPS, h, xq, a)
    w.w4a16_add_rmsnorm_i8(w.W4A16_BF16, x2, res, T, N, wt, EPS, x2, xq2, a2)
    assert torch.equal(xq, xq2) and torch.equal(a, a2) and torch.equal(x2, h)


@pytest.mark.parametrize("T,N", [(6, 512), (1100, 512), (6, 9008)])
def test_rows_that_are_not_finite_stay_their_own(T, N):
    x, res, wt = data(T, N, "bf16", 9)
    act = w.W4A16_BF16
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[1, 4, 5]] = True
    out = []
    for hurt in (False, True):
        if hurt:
            x[1, 3], x[4, N - 1], res[5, 100] = float("inf"), float("nan"), float("-inf")
        y, xq, a = torch.empty((T, N), dtype=torch.bfloat16, device="cuda"), torch.empty((T, N), dtype=torch.int8, device="cuda"), \
            torch.empty(T, device="cuda")
        w.w4a16_add_rmsnorm(act, x.cuda(), res.cuda(), T, N, wt.cuda(), EPS, None, y)
        w.w4a16_add_rmsnorm_i8(act, x.cuda(), res.cuda(), T, N, wt.cuda(), EPS, None, xq, a)
        out.append((y.cpu(), xq.cpu(), a.cpu()))
    for clean, dirty in zip(*out):
        assert torch.equal(clean[~bad], dirty[~bad])
    assert out[1][2][bad].isnan().all() and (out[1][1][bad] == 0).all()
    assert out[1][0][bad].isnan().any(1).all()


# ---- gradients ----------------------------------------------------------------------------------

def gradients(dy, dh, h, wt, eps=EPS):
    """The formulas in 64 bits, and what bounds the sums in them: sum |g h| and sum |dy h r|."""
    h, dy = h.double(), dy.double()
    N = h.shape[1]
    r = 1 / torch.sqrt((h * h).sum(1, keepdim=True) / N + eps)
    g = dy if wt is None else dy * wt.double()
    c = (g * h).sum(1, keepdim=True) * r * r / N
    dx = r * (g - h * c)
    mag = r * g.abs() + (r ** 3 / N) * h.abs() * (g * h).abs().sum(1, keepdim=True)
    if dh is not None:
        dx = dx + dh.double()
        mag = mag + dh.double().abs()
    term = dy * h * r
    return dx, term.sum(0), mag, term.abs().sum(0)


GRADS = [(1, 1), (1, 4096), (3, 7), (77, 500), (6, 1001), (700, 2048), (600, 3000), (9, 8200), (13, 12000), (5, 16384), (70, 33333), (1, 40001),
         (300, 17000)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,N", GRADS)
@pytest.mark.parametrize("with_dh,with_w", [(1, 1), (0, 0)])
def test_gradients(T, N, kind, with_dh, with_w):
    act, dt, u, tiny = TYPES[kind]
    h, dh, wt = data(T, N, kind, 11)
    dy = torch.randn((T, N), generator=torch.Generator().manual_seed(12)).to(dt)
    dh, wt = dh if with_dh else None, wt if with_w else None
    m = Arena()
    put = lambda t: None if t is None else m.put(t)
    dx, dw = m.out((T, N), dt), m.out((N,), torch.float32)
    nb = w.w4a16_add_rmsnorm_backward_workspace_bytes(T, N)
    args = put(dy), put(dh), put(h), T, N, put(wt), EPS
    ws = m.workspace(nb)
    w.w4a16_add_rmsnorm_backward(act, *args, dx, dw, ws, nb)
    ref, ref_w, mag, mag_w = gradients(dy, dh, h, wt)
    # sums of signed terms are off by their magnitudes' share; each result has at most eight roundings besides
    err = (dx.cpu().double() - ref).abs() - (u * ref.abs() + (1 + u) * (3 * REL(N) + 8 * F) * mag + tiny)
    assert err.max().item() <= 0
    err = (dw.cpu().double() - ref_w).abs() - (REL(N) + (T + 64) * F) * mag_w
    assert err.max().item() <= 0
    m.check()
    # either alone, and dx in dh's own array: the same bits
    if with_dh:
        own = args[1].clone()
        w.w4a16_add_rmsnorm_backward(act, args[0], own, *args[2:], own, None)
        assert torch.equal(own, dx)
    dw2 = m.out((N,), torch.float32)
    w.w4a16_add_rmsnorm_backward(act, *args, None, dw2, ws, nb)
    assert torch.equal(dw, dw2)
    m.check()


# the rows up to which one block writes the weight's gradient itself, and one more
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("T,N", [(16, 500), (17, 500), (8, 2048), (9, 2048), (4, 4000), (5, 4000), (2, 16384), (3, 16384), (2, 8192), (3, 8192)])
def test_gradients_of_few_rows(T, N, kind):
    test_gradients(T, N, kind, 1, 1)


# arrays from 32 MiB on, which pass the caches by: a wave a row up to sixteen, whole units and ragged rows
@pytest.mark.parametrize("T,N", [(35000, 496), (17000, 1001), (4300, 4000), (4200, 4097), (2100, 8176), (1100, 15600), (1101, 15601)])
def test_large_arrays(T, N):
    test_norm(T, N, "bf16", 1, 1, 1)
    test_gradients(T, N, "bf16", 1, 1)
    if N % 16 == 0:
        test_norm_i8(T, N, "bf16", 1, 1)


# one to sixteen waves a row and longer rows; one block, many, and arrays from 32 MiB on, in whole units and ragged rows; with
# eps = 0 and one that leaves a factor of 1 as it is (kernels of their own)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -60])
@pytest.mark.parametrize("kind,T,N", [
    ("bf16", 8, 496), ("f16", 17, 1001), ("f32", 77, 500), ("f32", 300, 17000), ("bf16", 2100, 20000), ("f16", 333, 33333),
    ("bf16", 35000, 496), ("f16", 17000, 1001), ("bf16", 4300, 4000), ("f16", 4200, 4097), ("bf16", 2100, 8176), ("f16", 1101, 15601),
    ("f32", 33000, 500), ("f32", 17000, 501), ("f32", 9001, 1000), ("f32", 4200, 2001), ("f32", 2300, 4000), ("f32", 1100, 8190)])
def test_gradient_of_the_weight_exactly(kind, T, N, eps):
    """Rows of +-1 have the factor 1, and whole numbers dy make each column's sum a whole number below 2^24,
    which any order of additions gives: a row lost or taken twice, in a block's rows or among the parts, shows."""
    act, dt = TYPES[kind][:2]
    g = torch.Generator(device="cuda").manual_seed(T + N)
    h = torch.randint(0, 2, (T, N), generator=g, device="cuda", dtype=torch.int8) * 2 - 1
    dy = torch.randint(-7, 8, (T, N), generator=g, device="cuda", dtype=torch.int8)
    ref = (h * dy).sum(0, dtype=torch.int64)
    dx, dw = torch.empty((T, N), dtype=dt, device="cuda"), torch.full((N,), float("nan"), device="cuda")
    ws, nb = w.alloc_add_rmsnorm_backward_workspace(T, N)
    w.w4a16_add_rmsnorm_backward(act, dy.to(dt), None, h.to(dt), T, N, None, eps, dx, dw, ws, nb)
    assert torch.equal(dw.double(), ref.double())


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -60])
def test_gradient_of_the_weight_past_32_bit_offsets(eps):
    N = 4096
    T = (1 << 31) // N + 5
    h = torch.ones((T, N), dtype=torch.bfloat16, device="cuda")
    dw, (ws, nb) = torch.empty(N, device="cuda"), w.alloc_add_rmsnorm_backward_workspace(T, N)
    w.w4a16_add_rmsnorm_backward(w.W4A16_BF16, h, None, h, T, N, None, eps, None, dw, ws, nb)
    assert (dw == T).all()


def check_gradients(kind, dy, h, wt, eps):
    act, dt, u, tiny = TYPES[kind]
    T, N = h.shape
    dx, dw = torch.empty((T, N), dtype=dt, device="cuda"), torch.empty(N, device="cuda")
    ws, nb = w.alloc_add_rmsnorm_backward_workspace(T, N)
    w.w4a16_add_rmsnorm_backward(act, dy.cuda(), None, h.cuda(), T, N, wt.cuda(), eps, dx, dw, ws, nb)
    ref, ref_w, mag, mag_w = gradients(dy, None, h, wt, eps)
    err = (dx.cpu().double() - ref).abs() - (u * ref.abs() + (1 + u) * (3 * REL(N) + 8 * F) * mag + tiny)
    assert not dx.isnan().any() and err.max().item() <= 0
    err = (dw.cpu().double() - ref_w).abs() - (REL(N) + (T + 64) * F) * mag_w
    assert not dw.isnan().any() and err.max().item() <= 0


SMALL = [("bf16", 512), ("f32", 500), ("bf16", 2048), ("f32", 8000), ("bf16", 15000), ("bf16", 20000), ("f32", 9001)]


@pytest.mark.parametrize("kind,N", SMALL)
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -109])
def test_gradients_of_rows_whose_factor_is_large(kind, N, eps):
    """Rows of +-2^-65: their squares and the sum of these are exact, their factor is 2^65 with eps = 0, and its square
    is past fp32's range."""
    dt = TYPES[kind][1]
    g = torch.Generator().manual_seed(41)
    h = (torch.randint(0, 2, (5, N), generator=g) * 2 - 1).float() * 2.0 ** -65
    dy, wt = torch.randn((5, N), generator=g), 1 + 0.3 * torch.randn(N, generator=g)
    check_gradients(kind, dy.to(dt), h.to(dt), wt.to(dt), eps)


def small_rows(kind, N):
    """Rows of magnitudes down to the type's smallest numbers."""
    e = torch.arange(-36, -128 if kind == "bf16" else -144, -4).double()
    x = torch.randn((len(e), N), generator=torch.Generator().manual_seed(42), dtype=torch.float64)
    return (x * torch.exp2(e)[:, None]).to(TYPES[kind][1])


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-30])
@pytest.mark.parametrize("kind,N", SMALL)
def test_gradients_of_rows_whose_squares_vanish(kind, N, eps):
    dt = TYPES[kind][1]
    h = small_rows(kind, N)
    g = torch.Generator().manual_seed(43)
    dy, wt = torch.randn(h.shape, generator=g) * 2.0 ** -20, 1 + 0.3 * torch.randn(N, generator=g)
    check_gradients(kind, dy.to(dt), h, wt.to(dt), float(np.float32(eps)))


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-30])
@pytest.mark.parametrize("kind,N", [("bf16", 16), ("f32", 496), ("bf16", 2048), ("f32", 8000), ("bf16", 20000), ("f32", 9001)])
def test_rows_whose_squares_vanish(kind, N, eps):
    """Squares below fp32's smallest numbers enter the sum all the same."""
    act, dt, u, _ = TYPES[kind]
    x, eps = small_rows(kind, N), float(np.float32(eps))
    T = x.shape[0]
    wt = (1 + 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(44))).to(dt)
    _, v = reference(x, None, wt, eps)
    small = 2.0 ** -149  # (values below fp32's normal numbers: half a step of these, and of the type's)
    y = x.cuda()
    h = torch.empty_like(y)
    w.w4a16_add_rmsnorm(act, y, None, T, N, wt.cuda(), eps, h, y)
    assert torch.equal(h.cpu(), x)
    least = torch.finfo(dt).smallest_normal * 2 * u + small
    assert not y.isnan().any() and ((y.cpu().double() - v).abs() <= (u + (1 + u) * REL(N)) * v.abs() + least).all()
    if N % 16:
        return
    xq, a = torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    h = x.cuda()
    w.w4a16_add_rmsnorm_i8(act, h, None, T, N, wt.cuda(), eps, h, xq, a)
    assert torch.equal(h.cpu(), x)
    top, a64 = v.abs().amax(1), a.cpu().double()
    normal = top > 2.0 ** -110
    assert ((a64 - top / 127).abs() <= (REL(N) + 2 * F) * top / 127)[normal].all()
    err = (xq.cpu().double() * a64[:, None] - v).abs() - (a64[:, None] * (0.5 + 128 * 2 * F) + REL(N) * v.abs())
    assert err[normal].max().item() <= 0


@pytest.mark.parametrize("T,N", [(3, 24), (2, 33)])
def test_gradients_against_differences(T, N):
    """Of L = sum(y dy) + sum(h dh) by the formulas in 64 bits: central differences with a step of 2^-12 are off by
    step^2 / 6 times the third derivative, below 1e-4 here (rows of magnitude one), and rounding, 1e-11."""
    g = torch.Generator().manual_seed(13)
    x, res, dy, dh = (torch.randn((T, N), generator=g) for _ in range(4))
    wt = 1 + 0.3 * torch.randn(N, generator=g)
    h, y = torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    w.w4a16_add_rmsnorm(w.W4A16_FP32, x.cuda(), res.cuda(), T, N, wt.cuda(), EPS, h, y)
    dx, dw = torch.empty_like(h), torch.empty(N, device="cuda")
    ws, nb = w.alloc_add_rmsnorm_backward_workspace(T, N)
    w.w4a16_add_rmsnorm_backward(w.W4A16_FP32, dy.cuda(), dh.cuda(), h, T, N, wt.cuda(), EPS, dx, dw, ws, nb)

    def loss(s, wt):
        return ((s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * wt * dy.double()).sum() + (s * dh.double()).sum()).item()

    step = 2.0 ** -12
    s = h.cpu().double()
    for t in range(T):
        for n in range(N):
            d = torch.zeros_like(s)
            d[t, n] = step
            diff = (loss(s + d, wt.double()) - loss(s - d, wt.double())) / (2 * step)
            assert abs(dx[t, n].item() - diff) <= 1e-4
    for n in range(N):
        d = torch.zeros(N, dtype=torch.float64)
        d[n] = step
        diff = (loss(s, wt.double() + d) - loss(s, wt.double() - d)) / (2 * step)
        assert abs(dw[n].item() - diff) <= 1e-4


def test_captured_training_step():
    """Forward and backward captured into a graph and replayed on new data, with eager calls between."""
    act, dt = w.W4A16_BF16, torch.bfloat16
    T, N = 300, 2048
    x, res, dy, dh, h, y, dx = (torch.empty((T, N), dtype=dt, device="cuda") for _ in range(7))
    wt, dw = torch.empty(N, dtype=dt, device="cuda"), torch.empty(N, device="cuda")
    ws, nb = w.alloc_add_rmsnorm_backward_workspace(T, N)

    def step():
        w.w4a16_add_rmsnorm(act, x, res, T, N, wt, EPS, h, y)
        w.w4a16_add_rmsnorm_backward(act, dy, dh, h, T, N, wt, EPS, dx, dw, ws, nb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, res, dy, dh):
            t.copy_(torch.randn((T, N), generator=g, device="cuda"))
        wt.copy_(torch.randn(N, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, y, dx, dw)]
        for t in (h, y, dx, dw):
            t.fill_(0)
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, y, dx, dw)))


def test_another_stream():
    T, N = 64, 4096
    x, res, wt = (t.cuda() for t in data(T, N, "f16", 15))
    ref, y = torch.empty_like(x), torch.empty_like(x)
    w.w4a16_add_rmsnorm(w.W4A16_FP16, x, res, T, N, wt, EPS, None, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    w.w4a16_add_rmsnorm(w.W4A16_FP16, x, res, T, N, wt, EPS, None, y, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements: the last rows against 64 bits (a call of other sizes may add in another order)."""
    N = 4096
    T = (1 << 31) // N + 5
    act, dt, u = w.W4A16_BF16, torch.bfloat16, 2.0 ** -8
    x = torch.empty((T, N), dtype=dt, device="cuda")
    x[-8:] = torch.randn((8, N), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x[:-8] = 1.0
    y, xq, a = torch.empty_like(x), torch.empty((T, N), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    w.w4a16_add_rmsnorm(act, x, None, T, N, None, EPS, None, y)
    w.w4a16_add_rmsnorm_i8(act, x, None, T, N, None, EPS, None, xq, a)
    last = x[-8:].cpu()
    _, v = reference(last, None, None)
    assert ((y[-8:].cpu().double() - v).abs() <= (u + (1 + u) * REL(N)) * v.abs()).all()
    a8, ref = a[-8:].cpu().double(), v.abs().amax(1) / 127
    assert ((a8 - ref).abs() <= (REL(N) + 2 * F) * ref).all()
    assert ((xq[-8:].cpu().double() * a8[:, None] - v).abs() <= a8[:, None] * (0.5 + 128 * 2 * F) + REL(N) * v.abs()).all()
    assert (y[0] == 1).all() and (xq[:-8] == 127).all()
    nb = w.w4a16_add_rmsnorm_backward_workspace_bytes(T, N)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(N, device="cuda")
    w.w4a16_add_rmsnorm_backward(act, x, None, x, T, N, None, EPS, dx, dw, ws, nb)
    ref, _, mag, _ = gradients(last, None, last, None)
    assert ((dx[-8:].cpu().double() - ref).abs() <= u * ref.abs() + (1 + u) * (3 * REL(N) + 8 * F) * mag).all()
