"""Products with 4-bit weights and group scales, called through the C ABI, against a plain float64
computation on the same inputs.

Tolerance, with u = 2^-24 and S_g the sum of a group's |code - zero| * |x|: the products are exact; the
tensor cores add 17 values at a time, each cut at 23 bits below the largest (17 * 2 u of what a step holds),
G / 16 steps a group; the groups' sums and the split of K are added in fp32, one rounding each, at most
K / G + 32 of them (fp32 rows: three column sums more).  So y is within
    (17 * G / 8 + K / G + 35) u  sum_g |scale_g| S_g,
then one rounding of half a step h.  For gate and up: SiLU's derivative is below 1.1, its own arithmetic
within 8 u.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


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


def matrix(E, R, K, G, scale_dtype, zeros, seed):
    g = gen(seed)
    q = torch.randint(0, 256, (E, R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((torch.rand((E, R, K // G), generator=g, device="cuda") + 0.5) * torch.where(
        torch.rand((E, R, K // G), generator=g, device="cuda") < 0.1, -0.03, 0.03)).to(scale_dtype)
    z = torch.randint(0, 16, (E, R, K // G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q, s, z


def dense(q, s, z):
    """[E][R][K] float64."""
    E, R, n = s.shape
    c = torch.stack((q & 15, q >> 4), -1).view(E, R, n, -1).double()
    return ((c - (8 if z is None else z.double().unsqueeze(-1))) * s.double().unsqueeze(-1)).view(E, R, -1)


def product(mat, x, start):
    """(y, sum of magnitudes) in float64."""
    W = dense(*mat)
    y, mag = (torch.zeros((x.shape[0], W.shape[1]), dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(W.shape[0]):
        a, b = start[e], start[e + 1]
        y[a:b] = x[a:b].double() @ W[e].t()
        mag[a:b] = x[a:b].double().abs() @ W[e].abs().t()
    return y, mag


def reference(mats, x, start, G):
    """(y, tolerance before the last rounding) in float64."""
    K = x.shape[1]
    y, mag = product(mats[0], x, start)
    err = (17 * G / 8 + K / G + 35) * U * mag
    if len(mats) == 2:
        u, umag = product(mats[1], x, start)
        uerr = (17 * G / 8 + K / G + 35) * U * umag
        s = y * torch.sigmoid(y)
        err = 1.1 * err * (u.abs() + uerr) + s.abs() * uerr + 8 * U * (s * u).abs()
        y = s * u
    return y, err


def segments(E, n, seed):
    """Offsets of n rows over E experts, some without a row."""
    if E == 1:
        return [0, n]
    cut = np.sort(np.random.default_rng(seed).integers(0, n + 1, E - 1))
    return [0, *cut.tolist(), n]


def close(got, ref, tol):
    d = (got.double() - ref).abs()
    assert torch.all(d <= tol), f"off by {float((d / tol.clamp(min=1e-300)).max()):.3g} tolerances"


CASES = [  # E, R, K, G, rows, dtype, scale dtype, zeros, pair
    (1, 1, 32, 32, 1, F32, F16, False, False), (1, 1, 64, 64, 2, BF16, BF16, True, True),
    (1, 17, 128, 128, 3, F16, F16, True, False), (1, 16, 96, 32, 1, BF16, BF16, False, False),
    (1, 100, 160, 32, 9, F16, BF16, True, True), (1, 7, 320, 64, 17, F32, F16, True, False),
    (1, 2048, 2048, 128, 1, BF16, F16, False, False), (1, 2048, 2048, 128, 1, F16, F16, False, False),
    (1, 333, 1152, 128, 33, F32, BF16, False, True), (1, 1000, 768, 32, 70, F16, F16, True, False),
    (1, 40, 32768, 32, 3, F32, F16, True, False), (1, 24, 32768, 128, 5, F16, F16, False, True),
    (1, 9, 20480, 64, 40, BF16, F16, True, False), (1, 5000, 512, 64, 4, F32, F16, False, False),
    (2, 64, 256, 32, 5, F32, F16, False, False), (5, 30, 416, 32, 64, BF16, BF16, True, True),
    (64, 96, 2048, 32, 64, F16, F16, False, True), (128, 128, 768, 64, 256, F32, F16, True, False),
    (7, 50, 128, 128, 300, F16, BF16, False, False), (1024, 8, 32, 32, 100, F16, F16, False, False),
    (3, 520, 640, 128, 2, BF16, F16, True, True), (300, 20, 192, 64, 40, F32, BF16, True, True),
    (16, 512, 1024, 64, 1, F16, F16, True, False), (4, 33, 8192, 32, 90, F32, F16, False, False),
]


@pytest.mark.parametrize("E,R,K,G,rows,dtype,sdtype,zeros,pair", CASES, ids=lambda v: str(v).replace("torch.", ""))
def test_product(ops, E, R, K, G, rows, dtype, sdtype, zeros, pair):
    mats = [matrix(E, R, K, G, sdtype, zeros, 1 + i) for i in range(1 + pair)]
    w = ops.MoeW4Weights(*mats[0], *(mats[1] if pair else ()))
    assert ops.moe_w4_weights_shape(w) == dict(E=E, R=R, K=K, group=G, pair=int(pair))
    start = segments(E, rows, K)
    behind = 2 if E > 1 else 0  # rows behind the last segment
    wide = torch.randn((rows + behind, K + 8), generator=gen(3), device="cuda").to(dtype)
    x = wide[:, :K]
    y = torch.full((rows + behind, R + 3), 5.0, dtype=dtype, device="cuda")
    es = None if E == 1 else torch.tensor(start, dtype=torch.int32, device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    ops.moe_w4_matvec(w, x, es, ws, y=y[:, :R])
    assert ops.moe_workspace_status(ws) == 0
    ref, err = reference(mats, x[:rows], start, G)
    close(y[:rows, :R], ref, err + HALF[dtype] * (ref.abs() + err) * 1.001 + TINY[dtype])
    assert torch.all(y[rows:] == 5.0) and torch.all(y[:, R:] == 5.0)
    if dtype is F32:  # held to single precision over the whole result as well
        rel = float((y[:rows, :R].double() - ref).norm() / ref.norm().clamp(min=1e-300))
        assert rel <= 1e-5, rel
    # contiguous rows (the wide loads) give the same bits
    assert torch.equal(ops.moe_w4_matvec(w, x[:rows].contiguous(), es, ws), y[:rows, :R])


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_rows_at_any_address_and_stride(ops, dtype):
    """Rows that 16-byte loads cannot take, one row for all (stride 0), and outputs at odd strides give the bits of
    contiguous ones."""
    mat = matrix(3, 50, 352, 32, F16, True, 1)
    w = ops.MoeW4Weights(*mat)
    es = torch.tensor([0, 4, 4, 21], dtype=torch.int32, device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    x = torch.randn((21, 352), generator=gen(2), device="cuda").to(dtype)
    want = ops.moe_w4_matvec(w, x, es, ws)
    for pad, shift in ((0, 1), (1, 0), (5, 3), (8, 8)):
        buf = torch.full((21 * (352 + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
        v = buf[shift:].view(21, 352 + pad)[:, :352]
        v.copy_(x)
        y = torch.empty((21, 50 + pad), dtype=dtype, device="cuda")[:, :50]
        assert torch.equal(ops.moe_w4_matvec(w, v, es, ws, y=y), want)
    one = x[:1].expand(21, 352)
    assert torch.equal(ops.moe_w4_matvec(w, one, es, ws), ops.moe_w4_matvec(w, one.contiguous(), es, ws))
    assert ops.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_a_row_does_not_depend_on_the_rows_beside_it(ops, dtype):
    """One matrix with and without offsets, and any number of rows at once: the same bits."""
    for R, K, G in ((2048, 2048, 128), (40, 640, 64), (20000, 256, 32)):
        w = ops.MoeW4Weights(*matrix(1, R, K, G, BF16, False, 1))
        ws = ops.new_sort_workspace(1, 1, 1)
        x = torch.randn((70, K), generator=gen(2), device="cuda").to(dtype)
        every = ops.moe_w4_matvec(w, x, None, ws)
        for a, b in ((0, 1), (3, 5), (0, 8), (10, 27), (31, 64)):
            assert torch.equal(ops.moe_w4_matvec(w, x[a:b], None, ws), every[a:b])
        y = torch.full_like(every, 5.0)
        ops.moe_w4_matvec(w, x, torch.tensor([0, 33], dtype=torch.int32, device="cuda"), ws, y=y)
        assert torch.equal(y[:33], every[:33]) and torch.all(y[33:] == 5.0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_rows_of_many_magnitudes(ops, dtype):
    """Values over 60 binades in one row: each is kept to 2^-22 of itself (bf16: exactly), or 2^-50 (2^-40) of the
    row's largest; the sums' own bound is test_product's."""
    R, K, G = 64, 512, 64
    mat = matrix(1, R, K, G, F16, False, 1)
    w = ops.MoeW4Weights(*mat)
    x = (torch.randn((6, K), generator=gen(2), device="cuda") * 2.0 ** torch.randint(-40, 20, (6, K), generator=gen(3), device="cuda").float()).to(dtype)
    x[5] = 0
    y = ops.moe_w4_matvec(w, x, None, ops.new_sort_workspace(1, 1, 1))
    ref, mag = product(mat, x, [0, 6])
    lost = torch.zeros_like(x, dtype=torch.float64)
    if dtype is F32:
        lost = torch.maximum(x.double().abs() * 2.0 ** -22, x.double().abs().amax(1, keepdim=True) * 2.0 ** -50)
    else:
        lost += x.double().abs().amax(1, keepdim=True) * 2.0 ** -40
    err = (17 * G / 8 + K / G + 35) * U * mag + lost @ dense(*mat)[0].abs().t()
    close(y, ref, err + HALF[dtype] * (ref.abs() + err) * 1.001 + TINY[dtype])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("K,rows", [(32, 1), (32, 37), (96, 7), (160, 33), (384, 20), (1024, 5), (4128, 3), (16416, 2)])
def test_powers_of_two_pass_through(ops, K, rows, dtype):
    """A row times a power of two gives its products times that power, bit for bit, whatever the rows beside it."""
    w = ops.MoeW4Weights(*matrix(1, 40, K, 32, F16, True, K))
    ws = ops.new_sort_workspace(1, 1, 1)
    x = torch.randn((rows, K), generator=gen(rows), device="cuda").to(dtype)
    power = torch.exp2(((torch.arange(rows, device="cuda") * 29) % 81 - 40).float()).unsqueeze(1)
    y = ops.moe_w4_matvec(w, x, None, ws)
    assert torch.equal(ops.moe_w4_matvec(w, (x * power).to(dtype), None, ws), (y * power).to(dtype))
    for j in range(rows):
        assert torch.equal(ops.moe_w4_matvec(w, x[j:j + 1], None, ws), y[j:j + 1])


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("G", [32, 64, 128])
def test_small_integers_are_exact(ops, G, dtype):
    """Codes, zero points and scales at their ends with integer rows: every sum is an integer below 2^24
    (below 2^8 steps of the type after a scale of 2^-k), so nothing may be lost but the last rounding."""
    E, R, K = 2, 24, 256
    q = torch.randint(0, 256, (E, R, K // 2), generator=gen(1), device="cuda", dtype=torch.uint8)
    q[0, 0], q[0, 1] = 0, 255
    z = torch.randint(0, 16, (E, R, K // G), generator=gen(2), device="cuda", dtype=torch.uint8)
    z[0, 0], z[0, 1] = 15, 0
    s = 2.0 ** torch.randint(-3, 3, (E, R, K // G), generator=gen(3), device="cuda").float()
    x = torch.randint(-8, 9, (11, K), generator=gen(4), device="cuda").to(dtype)
    ws = ops.new_sort_workspace(1, 1, 1)
    for zeros in (None, z):
        for sd in (F16, BF16):
            w = ops.MoeW4Weights(q, s.to(sd), zeros)
            start = [0, 4, 11]
            y = ops.moe_w4_matvec(w, x, torch.tensor(start, dtype=torch.int32, device="cuda"), ws)
            ref, _ = product((q, s.to(sd), zeros), x, start)
            assert torch.equal(y, ref.to(dtype))


def test_upper_bits_of_zero_points_are_ignored(ops):
    q, s, z = matrix(1, 20, 128, 32, F16, True, 1)
    x = torch.randn((2, 128), generator=gen(2), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    a, b = (ops.moe_w4_matvec(ops.MoeW4Weights(q, s, zz), x, None, ws) for zz in (z, z | 0xF0))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
def test_infinities_and_nan_stay_in_their_row(ops, dtype):
    """A row with an infinity or NaN has no effect on the others of its expert; large values of the type
    and its smallest do not turn into either."""
    q, s, _ = matrix(1, 48, 160, 32, F16, False, 1)
    q |= 0x99  # no code equals the zero point: an infinity always reaches the sum
    w = ops.MoeW4Weights(q, s)
    x = torch.randn((7, 160), generator=gen(2), device="cuda").to(dtype)
    ws = ops.new_sort_workspace(1, 1, 1)
    clean = ops.moe_w4_matvec(w, x, None, ws)
    bad = x.clone()
    bad[1, 5], bad[3, 150], bad[5, 159] = float("inf"), float("nan"), float("-inf")
    y = ops.moe_w4_matvec(w, bad, None, ws)
    assert torch.equal(y[[0, 2, 4, 6]], clean[[0, 2, 4, 6]])
    assert torch.all(torch.isnan(y[3]))
    sign = torch.sign(dense(q, s, None)[0])
    assert torch.equal(y[1], (float("inf") * sign[:, 5]).to(dtype))
    assert torch.equal(y[5], (float("-inf") * sign[:, 159]).to(dtype))
    big = torch.zeros((2, 160), dtype=dtype, device="cuda")
    big[0, 3] = torch.finfo(dtype).max / 16  # times a code less its zero point it has to stay in range
    big[1, 3] = torch.finfo(dtype).tiny
    small = ops.MoeW4Weights(q, torch.full_like(s, 2.0 ** -10))
    y = ops.moe_w4_matvec(small, big, None, ws)
    ref = big.double()[:, 3:4] * dense(q, torch.full_like(s, 2.0 ** -10), None)[0][:, 3]
    close(y, ref, (HALF[dtype] + 4 * U) * ref.abs() + TINY[dtype] * 2)


def test_bad_offsets_are_flagged_and_their_rows_left(ops):
    E, R, K = 4, 32, 64
    w = ops.MoeW4Weights(*matrix(E, R, K, 32, F16, False, 1))
    x = torch.randn((8, K), generator=gen(2), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    for start in ([1, 2, 4, 6, 8], [0, 5, 3, 6, 8], [0, 2, 4, 6, 9], [0, 2, 4, 2 ** 31 - 1, 8], [-3, 2, 4, 6, 8], [0, 2, -7, 6, 8]):
        es = torch.tensor(start, dtype=torch.int32, device="cuda")
        y = torch.full((8, R), 5.0, device="cuda")
        ops.moe_w4_matvec(w, x, es, ws, y=y)
        assert ops.moe_workspace_status(ws) == 2, start
        assert torch.all(y == 5.0)
    y = ops.moe_w4_matvec(w, x, torch.tensor([0, 0, 0, 0, 0], dtype=torch.int32, device="cuda"), ws,
                          y=torch.full((8, R), 5.0, device="cuda"))
    assert torch.all(y == 5.0) and ops.moe_workspace_status(ws) == 0


def test_decode_step_of_a_layer(ops):
    """Routing, sort, gate/up, down and unsort of a few tokens with 4-bit experts, against float64."""
    N, D, F, E, k = 5, 256, 128, 16, 4
    g = gen(3)
    x = torch.randn((N, D), generator=g, device="cuda")
    wr = torch.randn((E, D), generator=g, device="cuda") / 16
    gate, up = (matrix(E, F, D, 64, F16, True, s) for s in (1, 2))
    down = matrix(E, D, F, 32, F16, False, 3)
    gu, dn = ops.MoeW4Weights(*gate, *up), ops.MoeW4Weights(*down)
    ws = ops.new_workspace(N, D, E, F, k)
    r = ops.moe_router_topk(x, wr, None, k, True, ws)
    rows, start, _, _, tokRow = ops.moe_sort_tokens(x, r["topk_idx"], E, ws)
    y = ops.moe_w4_matvec(dn, ops.moe_w4_matvec(gu, rows, start, ws), start, ws)
    out = ops.moe_unsort_tokens(y, tokRow, r["topk_w"], ws)
    assert ops.moe_workspace_status(ws) == 0
    G, Up, Dn = (dense(*m) for m in (gate, up, down))
    ref = torch.zeros((N, D), dtype=torch.float64, device="cuda")
    for t in range(N):
        for s in range(k):
            e = int(r["topk_idx"][t, s])
            a, b = G[e] @ x[t].double(), Up[e] @ x[t].double()
            ref[t] += r["topk_w"][t, s].double() * (Dn[e] @ (a * torch.sigmoid(a) * b))
    # fp32 throughout: each of three chained products is within 1e-5 of its result (test_product)
    assert float((out.double() - ref).norm() / ref.norm()) <= 3e-5


def test_replayed_graph_and_two_streams(ops):
    E, R, K, n = 6, 200, 512, 24
    mat = matrix(E, R, K, 64, F16, True, 1)
    w = ops.MoeW4Weights(*mat)
    x = torch.randn((n, K), generator=gen(2), device="cuda").to(BF16)
    es = torch.tensor(segments(E, n, 1), dtype=torch.int32, device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    ops.moe_w4_matvec(w, x, es, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.moe_w4_matvec(w, x, es, ws)
    for seed in (5, 6):
        x.copy_(torch.randn((n, K), generator=gen(seed), device="cuda").to(BF16))
        es.copy_(torch.tensor(segments(E, n, seed), dtype=torch.int32, device="cuda"))
        graph.replay()
        assert torch.equal(y, ops.moe_w4_matvec(w, x, es, ws))
    # two calls at once on one handle, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [ops.new_sort_workspace(1, 1, 1) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, sp in zip(streams, spaces):
        with torch.cuda.stream(s):
            got += [ops.moe_w4_matvec(w, x, es, sp) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(t, got[0]) for t in got)


def test_refused_tensors(ops):
    q, s, z = matrix(2, 32, 128, 64, F16, True, 1)
    w = ops.MoeW4Weights(q, s, z)
    x, es = torch.randn((6, 128), device="cuda"), torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    for call in (lambda: ops.MoeW4Weights(q, s.float(), z), lambda: ops.MoeW4Weights(q.int(), s, z),
                 lambda: ops.MoeW4Weights(q, s, z[:, :, :1]), lambda: ops.MoeW4Weights(q, s[:, :, :1].expand(2, 32, 3)),
                 lambda: ops.MoeW4Weights(q, s, z, q, s.bfloat16(), z), lambda: ops.MoeW4Weights(q.cpu(), s, z),
                 lambda: ops.moe_w4_matvec(w, x[:, :64], es, ws), lambda: ops.moe_w4_matvec(w, x.double(), es, ws),
                 lambda: ops.moe_w4_matvec(w, x, es.long(), ws), lambda: ops.moe_w4_matvec(w, x, es[:2], ws),
                 lambda: ops.moe_w4_matvec(w, x.t().contiguous().t(), es, ws),
                 lambda: ops.moe_w4_matvec(w, x, es, ws, y=torch.empty((6, 32), device="cuda").half())):
        with pytest.raises(ValueError):
            call()
    both = torch.zeros((6, 160), device="cuda")
    for call, code in ((lambda: ops.MoeW4Weights(q, s, z, q, s), -1),                      # zero points on one side only
                       (lambda: ops.MoeW4Weights(q, s, None, q, s, z), -1),
                       (lambda: ops.MoeW4Weights(q, torch.ones((2, 32, 8), device="cuda").half()), -2),   # group 16
                       (lambda: ops.MoeW4Weights(q, torch.ones((2, 32, 1), device="cuda").half(),
                                                 None) and ops.moe_w4_matvec(w, x, None, ws), -1),        # offsets missing
                       (lambda: ops.moe_w4_matvec(w, x[:0], es, ws), -1),
                       (lambda: ops.moe_w4_matvec(w, x, es, ws[:128]), -3),
                       (lambda: ops.moe_w4_matvec(w, both[:, :128], es, ws, y=both[:, 120:152]), -1),     # overlap
                       (lambda: ops.moe_w4_matvec(w, x, es, ws, y=torch.empty((1, 32), device="cuda").expand(6, 32)), -1)):
        with pytest.raises(ops.MoeError) as err:
            call()
        assert err.value.code == code
    w.close()
    with pytest.raises(ValueError):
        ops.moe_w4_matvec(w, x, es, ws)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("largest", [1.0, 1.9921875, -1.5 * 2.0 ** -60, 2.0 ** 90])
def test_small_values_beside_a_large_one(ops, dtype, largest):
    """A value alone in the sum (weight 1), its row's largest at a weight of 0, over 60 binades: a bf16 value down to
    2^-31 of the largest is exact and a smaller one loses at most 2^-39 of it; an fp32 value at most 2^-22 of itself or
    2^-50 of the largest, and the last sum's rounding u.  (The bf16 results need no rounding: what is left of a value
    below 2^-31 of the largest are multiples of a step that is 2^-39 of it or more, at most 2^8 of them.)"""
    K = 64
    codes = torch.full((3, K), 8, dtype=torch.uint8, device="cuda")
    codes[0, 40] = codes[1, 5] = codes[2, 63] = 9
    w = ops.MoeW4Weights(codes[:, 0::2] | codes[:, 1::2] << 4, torch.ones((3, 2), device="cuda").half())
    e = torch.arange(-60, 1, device="cuda").float().repeat(40)
    m = 1 + torch.rand(e.shape, generator=gen(1), device="cuda")
    m[: 3 * 61] = torch.tensor([1.0, 1.5, 1.9921875], device="cuda").repeat_interleave(61)  # ties of the last steps
    v = (abs(largest) / 2 * m * torch.exp2(e)).to(dtype)  # below the largest
    v[::2] *= -1
    x = torch.zeros((v.numel(), K), dtype=dtype, device="cuda")
    x[:, 0] = largest
    x[:, 40], x[:, 5], x[:, 63] = v, v, v
    y = ops.moe_w4_matvec(w, x, None, ops.new_sort_workspace(1, 1, 1)).double()
    v, top = v.double().unsqueeze(1), abs(largest)
    if dtype is BF16:
        tol = torch.where(v.abs() >= top * 2.0 ** -31, 0.0, top * 2.0 ** -39)
    else:
        tol = torch.maximum(v.abs() * 2.0 ** -22, torch.full_like(v, top * 2.0 ** -50)) + U * 1.001 * v.abs()
    assert torch.all((y - v).abs() <= tol)


def far_scales(mat, scale, seed):
    """The matrix with bf16 scales of magnitude 0.5 .. 1.5 times `scale` (a number, or one per weight row)."""
    q, s, z = mat
    g = gen(seed)
    v = (torch.rand(s.shape, generator=g, device="cuda", dtype=torch.float64) + 0.5) * torch.sign(s).double()
    return q, (v * scale).float().to(BF16), z


def far_close(y, x, mats, start, G, dtype):
    """test_product's tolerance, and what the smallest fp32 numbers add: each of the K / G + 35 sums is off by up to
    2^-150, 2^13 times that where the row's largest passes 2^115; compared where no sum can leave fp32's range."""
    ref, err = reference(mats, x, start, G)
    small = x.double().abs().amax(1, keepdim=True) < 2.0 ** 115
    step = torch.where(small, 2.0 ** -13, 1.0).double() * 2.0 ** -137  # in float64: 2^-150 is 0 in fp32
    err = err + (x.shape[1] / G + 35) * step
    inside = product(mats[0], x, start)[1] < 2.0 ** 125
    assert torch.all(torch.isfinite(y[inside])) and int(inside.sum()) > 0
    tol = err + HALF[dtype] * (ref.abs() + err) * 1.001 + TINY[dtype]
    close(torch.where(inside, y.double(), 0.0), torch.where(inside, ref, 0.0), tol)
    return ref[inside]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("E,R,K,G,rows,zeros", [(1, 40, 256, 32, 1, False), (1, 33, 1280, 128, 20, True),
                                                (3, 24, 160, 32, 25, True), (2, 50, 384, 64, 9, False)])
@pytest.mark.parametrize("scale,value", [(100, -110), (125, -128), (-120, 100), (-125, 124), (60, -125), (-60, 60),
                                         (-10, 120)])
def test_scales_over_all_of_bf16(ops, scale, value, E, R, K, G, rows, zeros, dtype):
    """Large scales with small rows and small scales with large rows: finite wherever the definition's sums are."""
    mat = far_scales(matrix(E, R, K, G, BF16, zeros, 1), 2.0 ** scale, 2)
    w = ops.MoeW4Weights(*mat)
    start = segments(E, rows, K)
    es = None if E == 1 else torch.tensor(start, dtype=torch.int32, device="cuda")
    x = (torch.randn((rows, K), generator=gen(3), device="cuda", dtype=torch.float64) * 2.0 ** value).float().to(dtype)
    y = ops.moe_w4_matvec(w, x, es, ops.new_sort_workspace(1, 1, 1))
    assert float(far_close(y, x, [mat], start, G, dtype).abs().max()) > 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_scales_and_rows_of_many_magnitudes_together(ops, dtype):
    """A power of two for each weight row and for each activation row, from one end of the types to the other; a
    matrix of ordinary scales in the same handle keeps the bits that it has without the others."""
    R, K, G, rows = 57, 320, 32, 38
    near = matrix(1, R, K, G, BF16, True, 1)
    power = torch.arange(R, device="cuda", dtype=torch.float64) * 4 - 112
    far = far_scales(near, torch.exp2(power).view(1, R, 1), 2)
    both = [torch.cat((a, b)) for a, b in zip(near, far)]
    start = [0, rows, 2 * rows]
    x = torch.randn((rows, K), generator=gen(3), device="cuda", dtype=torch.float64)
    x = (x * torch.exp2(torch.arange(rows, device="cuda").double().view(-1, 1) * 6 - 112)).float().to(dtype)
    x = torch.cat((x, x))
    ws, es = ops.new_sort_workspace(1, 1, 1), torch.tensor(start, dtype=torch.int32, device="cuda")
    y = ops.moe_w4_matvec(ops.MoeW4Weights(*both), x, es, ws)
    far_close(y, x, [both], start, G, dtype)
    plain = ops.moe_w4_matvec(ops.MoeW4Weights(*(torch.cat((a, a)) for a in near)), x, es, ws)
    assert torch.equal(plain[4:rows], y[4:rows])  # from rows of 2^-88 on, where no sum nears the smallest numbers


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_gate_and_up_of_far_scales(ops, dtype):
    R, K, G, rows = 40, 256, 64, 11
    gate = far_scales(matrix(1, R, K, G, BF16, False, 1), 2.0 ** 98, 2)
    up = far_scales(matrix(1, R, K, G, BF16, False, 4), 2.0 ** 120, 5)
    x = (torch.randn((rows, K), generator=gen(3), device="cuda", dtype=torch.float64) * 2.0 ** -104).float().to(dtype)
    y = ops.moe_w4_matvec(ops.MoeW4Weights(*gate, *up), x, None, ops.new_sort_workspace(1, 1, 1))
    far_close(y, x, [gate, up], [0, rows], G, dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("rows", [1, 2, 13])
def test_rows_and_products_as_slices_of_one_buffer(ops, rows, dtype):
    """Columns side by side do not overlap, in either order or a row further on; one shared column does."""
    R, K = 48, 96
    w = ops.MoeW4Weights(*matrix(1, R, K, 32, F16, False, 1))
    ws = ops.new_sort_workspace(1, 1, 1)
    v = torch.randn((rows, K), generator=gen(2), device="cuda").to(dtype)
    want = ops.moe_w4_matvec(w, v, None, ws)
    for at, to, later in ((0, K, 0), (R, 0, 0), (R + 7, 3, 0), (0, K + 5, 0), (R, 0, 1), (0, K, 1)):
        buf = torch.full((rows + later, K + R + 16), 3.0, dtype=dtype, device="cuda")
        x, y = buf[:rows, at:at + K], buf[later:, to:to + R]
        x.copy_(v)
        left = torch.ones_like(buf, dtype=torch.bool)
        left[later:, to:to + R] = False
        kept = buf.clone()
        assert torch.equal(ops.moe_w4_matvec(w, x, None, ws, y=y), want)
        assert torch.equal(buf[left], kept[left])
    for at, to, later in ((0, K - 1, 0), (R - 1, 0, 0), (0, 0, 0)) + (((R - 1, 0, 1), (0, K - 1, 1)) if rows > 1 else ()):
        buf = torch.zeros((rows + later, K + R + 16), dtype=dtype, device="cuda")
        with pytest.raises(ops.MoeError) as err:
            ops.moe_w4_matvec(w, buf[:rows, at:at + K], None, ws, y=buf[later:, to:to + R])
        assert err.value.code == -1
