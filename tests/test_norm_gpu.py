"""Layer norm, its gradients and RMSNorm's, called through the C ABI, against plain float64 on the same inputs.

Tolerances, with u = 2^-24.  A row's sums take at most 16 additions in a thread, 5 in its warp, 16 over the warps
and 4 over a cluster: below 45 u of the sum of magnitudes.  So the mean is off by dm = 45 u mean|x|; the variance,
summed from deviations off by dm each (whose own sum stays below dm D), by 50 u of itself and dm^2; r by half of that and
4 u: rel_r = 30 u + (dm r)^2; h = (x - m) r by E_h = r dm + |h| (rel_r + 3 u).  The column sums add at most
N / 152 rows in a thread (a CTA's rows are dealt over the SMs), 16 groups, 20 partial sums a warp and 16 warps: n_c = N / 152 + 64.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_top_gb300 import build, ops as _ops

    build.build()
    torch.cuda.set_device(0)
    return _ops


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(N, D, dtype, seed, pad=0, at=0, off=0.3, level=1.0):
    """Rows of different level, off centre, `pad` elements apart, `at` elements into their buffer."""
    g = gen(seed)
    wide = torch.full((N * (D + pad) + at,), 7.0, dtype=dtype, device="cuda")
    x = wide[at:].view(N, D + pad)[:, :D]
    lv = level * torch.exp(0.5 * torch.randn((N, 1), generator=g, device="cuda"))
    x.copy_(((torch.randn((N, D), generator=g, device="cuda") + off) * lv).to(dtype))
    return x


def statistics(x, rms, eps):
    x = x.double()
    m = torch.zeros_like(x[:, :1]) if rms else x.mean(dim=1, keepdim=True)
    d = x - m
    r = 1 / torch.sqrt(d.square().mean(dim=1, keepdim=True) + eps)
    dm = torch.zeros_like(m) if rms else 45 * U * x.abs().mean(dim=1, keepdim=True)
    h = d * r
    rel = 30 * U + (dm * r) ** 2
    return h, r, dm, rel, r * dm + h.abs() * (rel + 3 * U)


def close(got, ref, tol, dtype=F32):
    d = (got.double() - ref).abs()
    tol = tol + HALF[dtype] * (ref.abs() + tol) + TINY[dtype]
    assert torch.all(d <= tol), f"off by {float((d / tol).max()):.3g} tolerances"


SHAPES = [  # N, D, pad, first element
    (1, 1, 0, 0), (3, 1, 0, 0), (2, 2, 0, 0), (5, 7, 0, 0), (1, 8, 0, 0), (4, 2048, 0, 0), (1, 2048, 8, 0),
    (33, 64, 0, 0), (1000, 100, 0, 0), (517, 1001, 0, 0), (517, 1001, 7, 1), (300, 2050, 0, 0), (7, 4096, 0, 8),
    (9, 8192, 0, 0), (3, 8193, 0, 0), (5, 8200, 0, 0), (2, 16384, 0, 0), (1, 32768, 0, 0), (3, 32767, 0, 0), (4, 20000, 8, 0),
    (2000, 512, 8, 0), (5000, 24, 0, 0), (700, 3000, 0, 2),
]


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("N,D,pad,at", SHAPES)
def test_layernorm(ops, N, D, pad, at, dtype):
    x = rows(N, D, dtype, 1, pad, at)
    gamma, beta = torch.randn(D, generator=gen(2), device="cuda"), torch.randn(D, generator=gen(3), device="cuda")
    for b in (beta, None):
        out = torch.full((N, D + 3), 5.0, dtype=dtype, device="cuda")
        y = ops.moe_layernorm(x, gamma, b, EPS, y=out[:, :D]) if pad else ops.moe_layernorm(x, gamma, b, EPS)
        h, r, dm, rel, e_h = statistics(x, False, EPS)
        ref = h * gamma.double() + (0 if b is None else b.double())
        tol = gamma.double().abs() * e_h + 2 * U * ((h * gamma.double()).abs() + (0 if b is None else b.double().abs()))
        close(y, ref, tol, dtype)
        assert torch.all(out[:, D:] == 5)


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("N,D,pad,at", SHAPES)
def test_gradients(ops, N, D, pad, at, dtype, rms):
    x, dy = rows(N, D, dtype, 4, pad, at), rows(N, D, dtype, 5, pad, at, off=0.05)
    gamma = torch.randn(D, generator=gen(6), device="cuda")
    ws = ops.new_norm_workspace(N, D)
    out = torch.full((N, D + 5), 5.0, dtype=dtype, device="cuda")
    to = out[:, :D] if pad else None
    if rms:
        d_x, d_gamma = ops.moe_rmsnorm_grad(dy, x, gamma, EPS, ws, d_x=to)
        d_beta = None
    else:
        d_x, d_gamma, d_beta = ops.moe_layernorm_grad(dy, x, gamma, EPS, ws, d_x=to)
    h, r, dm, rel, e_h = statistics(x, rms, EPS)
    d, gm = dy.double(), gamma.double()
    g = d * gm
    gd = (g * h / r).abs().sum(dim=1, keepdim=True)
    mgh, mg = (g * h).mean(dim=1, keepdim=True), torch.zeros_like(r) if rms else g.mean(dim=1, keepdim=True)
    e_mgh = r / D * (47 * U * gd + g.abs().sum(dim=1, keepdim=True) * dm) + mgh.abs() * (rel + 2 * U)
    inner = g - mg - h * mgh
    tol = r * (46 * U * g.abs().mean(dim=1, keepdim=True) + h.abs() * e_mgh + mgh.abs() * e_h +
               4 * U * (g.abs() + mg.abs() + (h * mgh).abs())) + (r * inner).abs() * (rel + 2 * U)
    close(d_x, r * inner, tol, dtype)
    n_c = N / 152 + 64
    close(d_gamma, (d * h).sum(0), (d.abs() * e_h).sum(0) + n_c * U * (d * h).abs().sum(0))
    if not rms:
        close(d_beta, d.sum(0), n_c * U * d.abs().sum(0))
        first = d_x.clone()  # the same places again: the order of a sum depends on how they are aligned
        again = ops.moe_layernorm_grad(dy, x, gamma, EPS, ws, d_x=d_x, beta=False)
        d_x = first
        assert again[2] is None and torch.equal(again[0], d_x) and torch.equal(again[1], d_gamma)
    assert torch.all(out[:, D:] == 5)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("D", [1, 2, 3, 7, 62, 127, 129, 255, 1000, 1027, 2046, 2048, 4381, 8191])
def test_layernorm_of_rows_at_any_place(ops, D, dtype):
    """x and y each at places of their own, many rows; nothing between y's rows is touched.  Bounds as in test_layernorm."""
    N = 1300
    gamma, beta = torch.randn(D, generator=gen(2), device="cuda"), torch.randn(D, generator=gen(3), device="cuda")
    for pads, ats, b in (((5, 1), (1, 3), beta), ((0, 2), (0, 6), None), ((9, 8), (7, 2), beta)):
        x = rows(N, D, dtype, 4, pads[0], ats[0])
        buf = torch.full((N * (D + pads[1]) + ats[1] + 9,), 5.0, dtype=dtype, device="cuda")
        wide = buf[ats[1]:ats[1] + N * (D + pads[1])].view(N, D + pads[1])
        y = ops.moe_layernorm(x, gamma, b, EPS, y=wide[:, :D])
        h, r, dm, rel, e_h = statistics(x, False, EPS)
        ref = h * gamma.double() + (0 if b is None else b.double())
        tol = gamma.double().abs() * e_h + 2 * U * ((h * gamma.double()).abs() + (0 if b is None else b.double().abs()))
        close(y, ref, tol, dtype)
        assert torch.all(wide[:, D:] == 5) and torch.all(buf[:ats[1]] == 5) and torch.all(buf[-9:] == 5)


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("D", [1, 2, 3, 5, 9, 63, 126, 127, 129, 130, 255, 1000, 1027, 2046, 2048, 2050, 4099, 4381, 8191])
def test_gradients_of_rows_at_any_place(ops, D, dtype, rms):
    """x, d_y and d_x each at places of their own, rows an odd number of elements apart; nothing between d_x's rows is
    touched.  Bounds as in test_gradients."""
    N = 67 if D > 1000 else 1500
    gamma = torch.randn(D, generator=gen(6), device="cuda")
    ws = ops.new_norm_workspace(N, D)
    for pads, ats in (((5, 3, 1), (1, 2, 3)), ((0, 7, 2), (0, 5, 6)), ((9, 8, 7), (7, 4, 2))):
        x, dy = rows(N, D, dtype, 4, pads[0], ats[0]), rows(N, D, dtype, 5, pads[1], ats[1], off=0.05)
        buf = torch.full((N * (D + pads[2]) + ats[2] + 9,), 5.0, dtype=dtype, device="cuda")
        wide = buf[ats[2]:ats[2] + N * (D + pads[2])].view(N, D + pads[2])
        if rms:
            d_x, d_gamma = ops.moe_rmsnorm_grad(dy, x, gamma, EPS, ws, d_x=wide[:, :D])
        else:
            d_x, d_gamma, d_beta = ops.moe_layernorm_grad(dy, x, gamma, EPS, ws, d_x=wide[:, :D])
        h, r, dm, rel, e_h = statistics(x, rms, EPS)
        d, gm = dy.double(), gamma.double()
        g = d * gm
        gd = (g * h / r).abs().sum(dim=1, keepdim=True)
        mgh, mg = (g * h).mean(dim=1, keepdim=True), torch.zeros_like(r) if rms else g.mean(dim=1, keepdim=True)
        e_mgh = r / D * (47 * U * gd + g.abs().sum(dim=1, keepdim=True) * dm) + mgh.abs() * (rel + 2 * U)
        inner = g - mg - h * mgh
        tol = r * (46 * U * g.abs().mean(dim=1, keepdim=True) + h.abs() * e_mgh + mgh.abs() * e_h +
                   4 * U * (g.abs() + mg.abs() + (h * mgh).abs())) + (r * inner).abs() * (rel + 2 * U)
        close(d_x, r * inner, tol, dtype)
        n_c = N / 152 + 64
        close(d_gamma, (d * h).sum(0), (d.abs() * e_h).sum(0) + n_c * U * (d * h).abs().sum(0))
        if not rms:
            close(d_beta, d.sum(0), n_c * U * d.abs().sum(0))
        assert torch.all(wide[:, D:] == 5) and torch.all(buf[:ats[2]] == 5) and torch.all(buf[-9:] == 5)
    one = rows(1, D, dtype, 18, 0, 3)  # a row for all, between values that are not finite
    around = torch.full((D + 32,), float("nan"), dtype=dtype, device="cuda")
    around[5:5 + D] = one[0]
    a = ops.moe_rmsnorm_grad(around[5:5 + D].unsqueeze(0).expand(N, D), x, gamma, EPS, ws, d_x=wide[:, :D])[0].clone()
    assert torch.equal(a, ops.moe_rmsnorm_grad(rows(N, D, dtype, 5, 3, 1).copy_(one.expand(N, D)), x, gamma, EPS, ws, d_x=wide[:, :D])[0])


def test_rows_far_off_centre(ops):
    """A mean of a thousand deviations, and one element a thousand times the others: the deviations keep their digits."""
    x = rows(64, 2048, F32, 7, off=1000.0)
    x[:, 0] = 3e6
    gamma = torch.ones(2048, device="cuda")
    y = ops.moe_layernorm(x, gamma, None, EPS)
    h, r, dm, rel, e_h = statistics(x, False, EPS)
    close(y, h, e_h + 2 * U * h.abs())


def test_constant_rows_zeros_and_one_column(ops):
    gamma, beta = torch.tensor([2.0, -3.0, 4.0, 0.5], device="cuda"), torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")
    x = torch.tensor([[5.0] * 4, [0.0] * 4], dtype=BF16, device="cuda")
    assert torch.equal(ops.moe_layernorm(x, gamma, beta, EPS), beta.to(BF16).expand(2, 4))
    ws = ops.new_norm_workspace(2, 4)
    d_x, d_gamma, d_beta = ops.moe_layernorm_grad(torch.ones_like(x), x, gamma, EPS, ws)
    assert torch.all(torch.isfinite(d_x.float())) and torch.equal(d_gamma, torch.zeros(4, device="cuda"))
    assert torch.equal(d_beta, torch.full((4,), 2.0, device="cuda"))
    d_x, d_gamma = ops.moe_rmsnorm_grad(torch.ones_like(x), torch.zeros_like(x), gamma, EPS, ws)
    ref = (gamma / torch.tensor(EPS, dtype=torch.float64).sqrt().item()).to(BF16)
    assert torch.allclose(d_x.float(), ref.float().expand(2, 4), rtol=2.0 ** -7) and torch.all(d_gamma == 0)


def test_nan_and_infinity_stay_in_their_rows(ops):
    x = rows(40, 512, F16, 8)
    gamma = torch.randn(512, generator=gen(9), device="cuda")
    dy = rows(40, 512, F16, 10)
    ws = ops.new_norm_workspace(40, 512)
    clean, clean_dx = ops.moe_layernorm(x, gamma, None, EPS), ops.moe_layernorm_grad(dy, x, gamma, EPS, ws)[0]
    x[3, 100], x[17, 0] = float("nan"), float("inf")
    y = ops.moe_layernorm(x, gamma, None, EPS)
    d_x, d_gamma, d_beta = ops.moe_layernorm_grad(dy, x, gamma, EPS, ws)
    keep = [i for i in range(40) if i not in (3, 17)]
    assert torch.equal(y[keep], clean[keep]) and torch.equal(d_x[keep], clean_dx[keep])
    assert torch.all(torch.isnan(y[3])) and torch.all(torch.isnan(d_x[3]))
    assert torch.all(torch.isfinite(d_beta)) and torch.all(torch.isnan(d_gamma))


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_against_differences(ops, rms):
    """Central differences of the forward calls in fp32 (step 2^-7, so a difference is off by 2^-7 squared times a third
    derivative of order one and by the results' roundings over the step: 1e-3 of the gradients' scale)."""
    N, D, step = 3, 24, 2.0 ** -7
    x = rows(N, D, F32, 11)
    x = x.clone()
    gamma, beta = torch.randn(D, generator=gen(12), device="cuda"), torch.randn(D, generator=gen(13), device="cuda")
    dy = torch.randn((N, D), generator=gen(14), device="cuda")
    ws = ops.new_norm_workspace(N, D)

    def loss(x, gamma, beta):
        y = ops.moe_rmsnorm(x, gamma, EPS) if rms else ops.moe_layernorm(x, gamma, beta, EPS)
        return float((y.double() * dy.double()).sum())

    got = ops.moe_rmsnorm_grad(dy, x, gamma, EPS, ws) if rms else ops.moe_layernorm_grad(dy, x, gamma, EPS, ws)
    args = [x, gamma] if rms else [x, gamma, beta]
    for a, g in zip(args, got):
        flat, grad = a.view(-1), g.reshape(-1)
        for i in range(0, flat.numel(), 5):
            keep = flat[i].item()
            flat[i] = keep + step
            up = loss(x, gamma, beta)
            flat[i] = keep - step
            down = loss(x, gamma, beta)
            flat[i] = keep
            assert abs((up - down) / (2 * step) - float(grad[i])) < 1e-3 * max(1.0, float(grad.abs().max()))


def test_one_gradient_row_for_all(ops):
    x = rows(50, 256, BF16, 15)
    gamma = torch.randn(256, generator=gen(16), device="cuda")
    one = torch.randn((1, 256), generator=gen(17), device="cuda").to(BF16)
    ws = ops.new_norm_workspace(50, 256)
    for a, b in zip(ops.moe_layernorm_grad(one.expand(50, 256), x, gamma, EPS, ws),
                    ops.moe_layernorm_grad(one.repeat(50, 1), x, gamma, EPS, ws)):
        assert torch.equal(a, b)


def test_captured_streams_and_repeats(ops):
    """The same bits from a graph, from another stream, and from a workspace of more rows."""
    x, dy = rows(900, 1024, BF16, 18), rows(900, 1024, BF16, 19)
    gamma, beta = torch.randn(1024, generator=gen(20), device="cuda"), torch.randn(1024, generator=gen(21), device="cuda")
    ws = ops.new_norm_workspace(900, 1024)
    y, grads = ops.moe_layernorm(x, gamma, beta, EPS), ops.moe_layernorm_grad(dy, x, gamma, EPS, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y2 = ops.moe_layernorm(x, gamma, beta, EPS)
        grads2 = ops.moe_layernorm_grad(dy, x, gamma, EPS, ws)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
    s = torch.cuda.Stream()
    big = ops.new_norm_workspace(5000, 1024)
    s.wait_stream(torch.cuda.current_stream())
    y3 = ops.moe_layernorm(x, gamma, beta, EPS, stream=s)
    grads3 = ops.moe_layernorm_grad(dy, x, gamma, EPS, big, stream=s)
    s.synchronize()
    assert torch.equal(y, y3) and all(torch.equal(a, b) for a, b in zip(grads, grads3))


def test_refusals(ops):
    x = rows(8, 64, BF16, 22)
    gamma = torch.ones(64, device="cuda")
    ws = ops.new_norm_workspace(8, 64)
    for bad in (lambda: ops.moe_layernorm(x, gamma, None, 0.0), lambda: ops.moe_layernorm(x, gamma, None, EPS, y=x),
                lambda: ops.moe_layernorm_grad(x, x, gamma, EPS, ws[:256]),
                lambda: ops.moe_layernorm_grad(x, x, gamma, float("nan"), ws),
                lambda: ops.moe_rmsnorm_grad(x, x, gamma, EPS, ws, d_x=x),
                lambda: ops.moe_layernorm(torch.zeros((1, 32769), device="cuda"), torch.ones(32769, device="cuda"), None, EPS)):
        with pytest.raises(ops.MoeError):
            bad()
    for bad in (lambda: ops.moe_layernorm(x, gamma.half(), None, EPS), lambda: ops.moe_layernorm(x.t(), torch.ones(8, device="cuda"), None, EPS),
                lambda: ops.moe_layernorm_grad(x.float(), x, gamma, EPS, ws), lambda: ops.moe_layernorm(x, gamma[:32], None, EPS),
                lambda: ops.moe_layernorm(x.cpu(), gamma, None, EPS)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("D", [256, 1001, 2046, 9000, 20001])
def test_layernorm_of_one_row_for_all(ops, D, dtype):
    """x with row stride 0: the bits of rows written out (which lie on the same boundaries)."""
    x = rows(1, D, dtype, 23)
    gamma, beta = torch.randn(D, generator=gen(24), device="cuda"), torch.randn(D, generator=gen(25), device="cuda")
    for N in (3, 700):
        y = ops.moe_layernorm(x.expand(N, D), gamma, beta, EPS)
        assert torch.equal(y, ops.moe_layernorm(x.repeat(N, 1), gamma, beta, EPS)) and torch.equal(y, y[:1].expand(N, D))


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("D", [8193, 12002, 16385, 32767])
def test_gradients_of_long_rows_at_any_place(ops, D, dtype, rms):
    """Rows longer than a tile of shared memory takes, more of them than CTAs, an odd number of elements apart.  Bounds as in
    test_gradients."""
    N = 700
    gamma = torch.randn(D, generator=gen(6), device="cuda")
    ws = ops.new_norm_workspace(N, D)
    for pads, at in (((0, 0, 0), 0), ((1, 5, 3), 3)):
        x, dy = rows(N, D, dtype, 26, pads[0], at), rows(N, D, dtype, 27, pads[1], at, off=0.05)
        buf = torch.full((N * (D + pads[2]) + at + 9,), 5.0, dtype=dtype, device="cuda")
        wide = buf[at:at + N * (D + pads[2])].view(N, D + pads[2])
        got = (ops.moe_rmsnorm_grad if rms else ops.moe_layernorm_grad)(dy, x, gamma, EPS, ws, d_x=wide[:, :D])
        h, r, dm, rel, e_h = statistics(x, rms, EPS)
        d, gm = dy.double(), gamma.double()
        g = d * gm
        mgh, mg = (g * h).mean(dim=1, keepdim=True), torch.zeros_like(r) if rms else g.mean(dim=1, keepdim=True)
        sizes = g.abs().sum(dim=1, keepdim=True)
        e_mgh = r / D * (47 * U * (g * h / r).abs().sum(dim=1, keepdim=True) + sizes * dm) + mgh.abs() * (rel + 2 * U)
        inner = g - mg - h * mgh
        tol = r * (46 * U * sizes / D + h.abs() * e_mgh + mgh.abs() * e_h + 4 * U * (g.abs() + mg.abs() + (h * mgh).abs()))
        close(got[0], r * inner, tol + (r * inner).abs() * (rel + 2 * U), dtype)
        n_c = N / 152 + 64
        close(got[1], (d * h).sum(0), (d.abs() * e_h).sum(0) + n_c * U * (d * h).abs().sum(0))
        if not rms:
            close(got[2], d.sum(0), n_c * U * d.abs().sum(0))
        assert torch.all(wide[:, D:] == 5) and torch.all(buf[:at] == 5) and torch.all(buf[-9:] == 5)
