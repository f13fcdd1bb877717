"""Products of 16-bit rows with 16-bit matrices (bias, activation, gate and up, residual; by expert), called through the
C ABI, against plain float64 on the same inputs.

Whole-number inputs have whole-number sums below 2^24, which every order of summation forms exactly: those results must
be the definition's, rounded once.  Tolerance elsewhere, with u = 2^-24: a tensor-core step adds 16 products to the sum
so far, each cut 23 bits below the largest: 17 * 2 u of it, K / 16 steps, and at most 16 more additions where warps share
a row; no partial sum of random signs exceeds B = 6 sqrt(sum (w x)^2).  So a sum is off by s = (K / 16 + 16) 34 u B.
Bias, product with up and residual round once each (u); the activations are within 2^-18 of their value and their
derivatives below 1.13.  Then half a step of the type.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
F16, BF16 = torch.float16, torch.bfloat16
ACT = {"none": lambda v: v, "relu": lambda v: torch.where(v < 0, torch.zeros_like(v), v), "silu": lambda v: v * torch.sigmoid(v),
       "gelu": lambda v: v * torch.special.ndtr(v)}


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixture_experts_ffn_top_gb300 import build, ops as _ops

    build.build()
    torch.cuda.set_device(0)
    return _ops


@pytest.fixture(scope="module")
def ws(ops):
    return ops.new_sort_workspace(1, 1, 1)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * scale).to(dtype)


def whole(shape, dtype, seed, top=3):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").to(dtype)


def strided(t, pad, at=0):
    """t's values in rows `pad` elements further apart, `at` elements into their buffer."""
    n, d = t.shape
    buf = torch.full((n * (d + pad) + at,), 9.0, dtype=t.dtype, device="cuda")
    v = buf[at:].view(n, d + pad)[:, :d]
    v.copy_(t)
    return v


def offsets(E, n, seed):
    """Offsets of n rows over E experts, some without a row."""
    if E == 1:
        return [0, n]
    cut = torch.randint(0, n + 1, (E - 1,), generator=gen(seed), device="cuda").sort().values
    return [0, *cut.tolist(), n]


def reference(x, w, start, w_up=None, bias=None, bias_up=None, act="none", residual=None):
    """(y, tolerance before the last rounding) in float64, over the rows of the segments."""
    K = x.shape[1]
    steps = (K / 16 + 16) * 34 * U
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = start[e], start[e + 1]
        if a == b:
            continue
        xe = x[a:b].double()

        def product(m, c):
            p = xe @ m[e].double().t()
            err = steps * 6 * torch.sqrt(xe.square() @ m[e].double().t().square())
            if c is not None:
                p = p + c[e].double()
                err = err + U * p.abs()
            return p, err

        v, err = product(w, bias)
        v, err = ACT[act](v), 1.13 * err
        err = err + (2.0 ** -18 * v.abs() if act in ("silu", "gelu") else 0)
        if w_up is not None:
            u, uerr = product(w_up, bias_up)
            err = err * (u.abs() + uerr) + v.abs() * uerr + U * (v * u).abs()
            v = v * u
        if residual is not None:
            v = v + residual[a:b].double()
            err = err + U * v.abs()
        y[a:b], tol[a:b] = v, err
    return y, tol


def close(got, ref, tol):
    d = (got.double() - ref).abs()
    tol = tol + HALF[got.dtype] * (ref.abs() + tol) + TINY[got.dtype]
    assert torch.all(d <= tol), f"off by {float((d / tol).max()):.3g} tolerances at {torch.nonzero(d > tol)[:4].tolist()}"


SIZES = [  # E, rows, R, K
    (1, 1, 1, 8), (1, 1, 16, 64), (1, 1, 2048, 2048), (1, 2, 17, 40), (1, 3, 700, 1032), (1, 8, 100, 2056), (1, 9, 33, 512),
    (1, 17, 130, 72), (1, 31, 513, 256), (1, 32, 300, 4096), (1, 5, 5, 16384), (1, 20, 4000, 24), (1, 32, 40, 9000),
    (1, 33, 1, 8), (1, 33, 257, 64), (1, 100, 300, 72), (1, 128, 256, 128), (1, 129, 130, 200), (1, 1000, 520, 1032),
    (1, 257, 2047, 264), (1, 4096, 96, 2048), (1, 640, 31, 64),
    (1, 8, 20000, 776), (1, 12, 9000, 520), (1, 4, 12000, 1016), (1, 6, 15000, 504), (2, 1, 40, 64), (5, 7, 30, 416), (64, 32, 96, 1024), (1024, 30, 8, 32), (3, 32, 520, 640), (16, 2, 512, 1024),
    (2, 40, 64, 256), (7, 300, 50, 128), (64, 500, 96, 512), (1024, 100, 8, 32), (1024, 5000, 24, 64), (3, 1000, 520, 640),
    (128, 4000, 130, 96), (300, 64, 20, 192),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("E,n,R,K", SIZES)
def test_whole_numbers(ops, ws, E, n, R, K, dtype):
    """Exact sums, every row and column: gate and up (sums times sums stay whole) and the single matrix."""
    start = offsets(E, n, K)
    behind = 3 if E > 1 else 0
    x = strided(whole((n + behind, K), dtype, 1, 1), 8)
    w, up = whole((E, R, K), dtype, 2, 1), whole((E, R, K), dtype, 3, 1)
    bias, res = whole((E, R), torch.float32, 4), whole((n + behind, R), dtype, 5)
    es = None if E == 1 else torch.tensor(start, dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(bias=bias, act="relu", residual=res), dict(w_up=up, bias_up=bias)):
        y = torch.full((n + behind, R + 1), 7.0, dtype=dtype, device="cuda")
        ops.moe_matmul(x, w, ws, expStart=es, y=y[:, :R], **kw)
        ref, _ = reference(x, w, start, **kw)
        assert torch.equal(y[:n, :R], ref[:n].to(dtype)), f"rows {torch.nonzero((y[:n, :R] != ref[:n].to(dtype)).any(1))[:8].tolist()}"
        assert torch.all(y[:, R:] == 7) and torch.all(y[n:] == 7)
    assert ops.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("E,n,R,K", [(1, 1, 2048, 2048), (1, 13, 100, 1000), (1, 300, 520, 1032), (6, 24, 96, 512), (6, 900, 200, 768)])
def test_epilogues(ops, ws, E, n, R, K, dtype, act):
    start = offsets(E, n, 7)
    es = None if E == 1 else torch.tensor(start, dtype=torch.int32, device="cuda")
    x, w, up = randn((n, K), dtype, 1), randn((E, R, K), dtype, 2, 2 * K ** -0.5), randn((E, R, K), dtype, 3, K ** -0.5)
    b, c, res = randn((E, R), torch.float32, 4), randn((E, R), torch.float32, 5), randn((n, R), dtype, 6)
    for kw in (dict(act=act), dict(act=act, bias=b, residual=res), dict(act=act, w_up=up), dict(act=act, w_up=up, bias=b, bias_up=c, residual=res),
               dict(act=act, w_up=up, bias_up=c)):
        y = ops.moe_matmul(x, w, ws, expStart=es, **kw)
        close(y, *reference(x, w, start, **kw))


def test_activations_over_their_range(ops, ws):
    """One column times one: the activations of values from the smallest to the largest, and of infinities."""
    v = torch.cat((torch.linspace(-30, 30, 4001), torch.tensor([0.0, -0.0, 1e-4, -1e-4, 87.0, -87.0, -88.5, -90.0, 1e4, -1e4, 6e4, -6e4]))).to(F16).cuda()
    for n in (v.numel(), 20):
        x = torch.zeros((n, 8), dtype=F16, device="cuda")
        x[:, 0] = v[-n:]
        w = torch.zeros((1, 1, 8), dtype=F16, device="cuda")
        w[..., 0] = 1
        for act in ("relu", "silu", "gelu"):
            ref = ACT[act](x[:, :1].double())
            close(ops.moe_matmul(x, w, ws, act=act), ref, 2.0 ** -18 * ref.abs() + 2.0 ** -126)
        x[0, 0], x[1, 0] = float("inf"), float("nan")
        for act in ("none", "relu", "silu", "gelu"):
            y = ops.moe_matmul(x, w, ws, act=act)
            assert torch.isposinf(y[0, 0]) and torch.isnan(y[1, 0]) and torch.all(torch.isfinite(y[2:]))


@pytest.mark.parametrize("n", [20, 200])
def test_nan_stays_in_its_row(ops, ws, n):
    x, w = randn((n, 512), BF16, 1), randn((4, 64, 512), BF16, 2)
    start = torch.tensor([0, n // 3, n // 3, n - 1, n], dtype=torch.int32, device="cuda")
    clean = ops.moe_matmul(x, w, ws, expStart=start)
    x[n // 3 - 1, 5], x[n - 1] = float("nan"), float("inf")
    y = ops.moe_matmul(x, w, ws, expStart=start)
    keep = [i for i in range(n) if i not in (n // 3 - 1, n - 1)]
    assert torch.equal(y[keep], clean[keep]) and torch.all(torch.isnan(y[n // 3 - 1]))


@pytest.mark.parametrize("n", [9, 150])
def test_residual_in_place_and_odd_places(ops, ws, n):
    """y at odd addresses and strides; the residual y itself; a residual row for all (stride 0)."""
    x, w = whole((n, 64), F16, 1), whole((1, 77, 64), F16, 2)
    ref = x.double() @ w[0].double().t()
    for pad, at in ((0, 0), (3, 1), (8, 8), (19, 5)):
        y = strided(whole((n, 77), F16, 3), pad, at)
        want = (ref + y.double()).to(F16)
        out = ops.moe_matmul(x, w, ws, residual=y, y=y)
        assert out is y and torch.equal(y, want)
    one = whole((1, 77), F16, 4)
    assert torch.equal(ops.moe_matmul(x, w, ws, residual=one.expand(n, 77)), (ref + one.double()).to(F16))


@pytest.mark.parametrize("n", [16, 64])
def test_bad_offsets(ops, ws, n):
    x, w = whole((n, 32), BF16, 1), whole((4, 16, 32), BF16, 2)
    for bad in ([1, 4, 8, 12, n], [0, 8, 4, 12, n], [0, 4, 8, 12, n + 1], [-1, 4, 8, 12, n], [0, n + 5, 8, 12, n]):
        y = torch.full((n, 16), 3.0, dtype=BF16, device="cuda")
        ops.moe_matmul(x, w, ws, expStart=torch.tensor(bad, dtype=torch.int32, device="cuda"), y=y)
        assert ops.moe_workspace_status(ws) == 2 and torch.all(y == 3)  # MOE_DEV_BAD_CSR
    y = torch.full((n, 16), 3.0, dtype=BF16, device="cuda")
    ops.moe_matmul(x, w, ws, expStart=torch.zeros(5, dtype=torch.int32, device="cuda"), y=y)
    assert ops.moe_workspace_status(ws) == 0 and torch.all(y == 3)


def test_captured_and_on_another_stream(ops, ws):
    for n in (3, 500):
        x, w, up = randn((n, 512), BF16, 1), randn((5, 300, 512), BF16, 2, 0.04), randn((5, 300, 512), BF16, 3, 0.04)
        start = torch.tensor(offsets(5, n, 1), dtype=torch.int32, device="cuda")
        y = ops.moe_matmul(x, w, ws, expStart=start, w_up=up, act="silu")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y2 = ops.moe_matmul(x, w, ws, expStart=start, w_up=up, act="silu")
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        y3 = ops.moe_matmul(x, w, ws, expStart=start, w_up=up, act="silu", stream=s)
        s.synchronize()
        assert torch.equal(y, y2) and torch.equal(y, y3)


def test_calls_at_once(ops, ws):
    """Few rows and many, on two streams at once: the same bits as alone."""
    w = randn((5, 700, 520), BF16, 2, 0.04)
    xs = [randn((n, 520), BF16, 1) for n in (24, 1500)]
    starts = [torch.tensor(offsets(5, x.shape[0], 1), dtype=torch.int32, device="cuda") for x in xs]
    want = [ops.moe_matmul(x, w, ws, expStart=s) for x, s in zip(xs, starts)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(i, torch.empty_like(want[i])) for _ in range(8) for i in (0, 1, 1)]
    torch.cuda.synchronize()
    for j, (i, y) in enumerate(outs):
        ops.moe_matmul(xs[i], w, ws, expStart=starts[i], y=y, stream=streams[j % 3])
    torch.cuda.synchronize()
    assert ops.moe_workspace_status(ws) == 0 and all(torch.equal(y, want[i]) for i, y in outs)


def test_large_offsets(ops, ws):
    """Results past 2^31 elements from the first."""
    n, R = 70000, 32768
    x, w = whole((n, 8), BF16, 1), whole((1, R, 8), BF16, 2)
    y = ops.moe_matmul(x, w, ws)
    for rows in (slice(0, 40), slice(65530, 65570), slice(n - 40, n)):
        assert torch.equal(y[rows], (x[rows].double() @ w[0].double().t()).to(BF16))


def test_refusals(ops, ws):
    x, w = randn((40, 64), BF16, 1), randn((1, 16, 64), BF16, 2)
    wide = randn((40, 65), BF16, 3)
    for bad in (lambda: ops.moe_matmul(wide[:, 1:], w, ws), lambda: ops.moe_matmul(x[:, :60], w[:, :, :60].contiguous(), ws),
                lambda: ops.moe_matmul(x, w, ws, y=x[:, :16]), lambda: ops.moe_matmul(x, w, ws, bias_up=torch.zeros((1, 16), device="cuda")),
                lambda: ops.moe_matmul(x, w.expand(2, 16, 64).contiguous(), ws), lambda: ops.moe_matmul(x, w, ws[:128]),
                lambda: ops.moe_matmul(x[:1].expand(40, 64), w, ws)):
        with pytest.raises(ops.MoeError):
            bad()
    for bad in (lambda: ops.moe_matmul(x.float(), w.float(), ws), lambda: ops.moe_matmul(x, w.half(), ws),
                lambda: ops.moe_matmul(x, w, ws, act="tanh"), lambda: ops.moe_matmul(x, w, ws, bias=torch.zeros(16, device="cuda")),
                lambda: ops.moe_matmul(x, w[:, :, :32], ws), lambda: ops.moe_matmul(x.cpu(), w, ws),
                lambda: ops.moe_matmul(x, w, ws, residual=x)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("n", [24, 2000])
def test_activations_of_bf16_over_their_range(ops, ws, n):
    """bf16 keeps the activations' far ends, down to 2^-126: SiLU's and GELU's values there are within 2^-15 (an exponent
    near 126 whose roundings of 2^-24 each count 87-fold in the result), then half a step; nothing below 2^-126 is asked
    for.  The normal distribution by erfc: 1 + erf has no digits left there."""
    act_of = dict(ACT, gelu=lambda v: 0.5 * v * torch.erfc(v * -(0.5 ** 0.5)))
    v = torch.cat((-torch.linspace(0, 120, 1500), torch.linspace(0, 120, 400), -torch.linspace(8, 14, 76),
                   torch.tensor([-86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -1e3, -1e5, -3e38, 1e5, 3e38, 1e-30, -1e-30, 2e-38, -2e-38, 0.0])))
    v = torch.cat((v, torch.zeros(2000 - v.numel()))).to(BF16).cuda()
    for lo in [0] if n == 2000 else range(1784, 2000, n):
        x = torch.zeros((n, 8), dtype=BF16, device="cuda")
        x[:, 0] = v[lo:lo + n]
        w = torch.zeros((1, 1, 8), dtype=BF16, device="cuda")
        w[..., 0] = 1
        for act in ("relu", "silu", "gelu"):
            ref = act_of[act](x[:, :1].double())
            close(ops.moe_matmul(x, w, ws, act=act), ref, 2.0 ** -15 * ref.abs() + 2.0 ** -126)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("E", [1, 2, 3])
@pytest.mark.parametrize("n", [9, 12, 16, 17, 24, 25, 31, 32])
def test_some_rows_of_few_matrices(ops, ws, n, E, dtype):
    """Where either kernel may serve, by the sizes of the matrices: the definition's results, with offsets (uneven ones,
    one matrix among them) and without, gate and up, rows behind the last segment left alone."""
    for R, K in ((40, 64), (2600, 72), (9000, 40)):
        x, w, up = whole((n + 2, K), dtype, 1, 1), whole((E, R, K), dtype, 2, 1), whole((E, R, K), dtype, 3, 1)
        for start in ([n * e // E for e in range(E + 1)], [0] + [n - 1] * (E - 1) + [n]):
            offsets_ = torch.tensor(start, dtype=torch.int32, device="cuda")
            for es, kw in ((offsets_, dict()), (offsets_, dict(w_up=up))) + (((None, dict()),) if E == 1 else ()):
                rows = x[:n] if es is None else x
                y = torch.full((rows.shape[0], R), 7.0, dtype=dtype, device="cuda")
                ops.moe_matmul(rows, w, ws, expStart=es, y=y, **kw)
                ref, _ = reference(rows, w, start, **kw)
                assert torch.equal(y[:n], ref[:n].to(dtype)) and torch.all(y[n:] == 7)
    assert ops.moe_workspace_status(ws) == 0
