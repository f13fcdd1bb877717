"""The whole layer for decode batches (router, top-k, 16-bit experts, shared expert, residual in one kernel), called
through the C ABI, against plain float64 on the same inputs.

Tolerance, with u = 2^-24.  Router: a logit's fp32 sum is off by e_l = (D / 256 + 24) u sum |W x| (a thread's products,
its warp, the warps), so a routing weight by 2 max e_l + 16 u of itself; tokens whose k-th and next logit lie closer
than twice that may choose either and are left out of random cases (they are made not to exist).  Gate, up and down: a
tensor-core step adds 16 products to the sum so far, each cut 23 bits below the largest (34 u of it), partial sums of
random signs stay below B = 6 sqrt(sum of squares): s = (K / 16 + 24) 34 u B.  h = w SiLU(gate) up carries the sums'
errors (SiLU's derivative is below 1.1), 8 u of its own, and enters the second product within 2^-17 of itself.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
F16, BF16 = torch.float16, torch.bfloat16


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


def layer(N, D, E, F, dtype, Fs=0, gated=False, seed=0, skew=0.0, h_scale=1.0):
    g = gen(seed)

    def rand(*shape, scale=1.0, of=dtype):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(of)

    s = {"x": rand(N, D), "routerW": rand(E, D, scale=D ** -0.5, of=torch.float32), "gate": rand(E, F, D, scale=D ** -0.5),
         "up": rand(E, F, D, scale=h_scale * D ** -0.5), "down": rand(E, D, F, scale=F ** -0.5 / h_scale), "shared": None, "shexp_gate": None}
    if skew:
        s["x"][:, D - 1] = 1
        s["routerW"][:, D - 1] = -skew * torch.log(torch.arange(E, device="cuda") + 1.0)
    if Fs:
        s["shared"] = (rand(Fs, D, scale=D ** -0.5), rand(Fs, D, scale=D ** -0.5), rand(D, Fs, scale=Fs ** -0.5))
        s["shexp_gate"] = rand(D, scale=D ** -0.5, of=torch.float32) if gated else None
    s["residual"] = rand(N, D)
    return s


def expert(x, gate, up, down, w, e_w):
    """(w down(SiLU(gate x) up x), its error's bound) for rows x and weights w [rows] known up to e_w relative."""
    D, F = gate.shape[1], gate.shape[0]
    gate, up, down, w = gate.double(), up.double(), down.double(), w.unsqueeze(1)
    s = (D / 16 + 24) * 34 * U * 6
    a, b = x @ gate.t(), x @ up.t()
    ea, eb = s * torch.sqrt(x.square() @ gate.t().square()), s * torch.sqrt(x.square() @ up.t().square())
    act = a * torch.sigmoid(a)
    h = w * act * b
    eh = w.abs() * (1.1 * ea * (b.abs() + eb) + act.abs() * eb) + h.abs() * (8 * U + e_w.unsqueeze(1) + 2.0 ** -17)
    y = h @ down.t()
    ey = eh @ down.t().abs() + (F / 16 + 24) * 34 * U * 6 * torch.sqrt(h.square() @ down.t().square())
    return y, ey


def reference(s, k, norm, residual=False):
    x = s["x"].double()
    N, D = x.shape
    l = x @ s["routerW"].double().t()
    e_l = ((D / 256 + 24) * U * (x.abs() @ s["routerW"].double().abs().t())).amax(dim=1)
    top, idx = torch.topk(l, min(k + 1, l.shape[1]), dim=1)
    if top.shape[1] > k:
        assert torch.all(top[:, k - 1] - top[:, k] > 2 * e_l), "a choice that rounding may turn: take another seed"
    idx = idx[:, :k]
    p = torch.softmax(l, dim=1).gather(1, idx)
    w = p / p.sum(dim=1, keepdim=True) if norm else p
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(N):
        for j in range(k):
            e = int(idx[t, j])
            a, b = expert(x[t:t + 1], s["gate"][e], s["up"][e], s["down"][e], w[t:t + 1, j], 2 * e_l[t:t + 1] + 16 * U)
            y[t] += a[0]
            tol[t] += b[0]
    if s["shared"] is not None:
        ws, ew = torch.ones(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
        if s["shexp_gate"] is not None:
            v = s["shexp_gate"].double()
            ws, ew = torch.sigmoid(x @ v), 8 * U + (D / 256 + 24) * U * (x.abs() @ v.abs())
        a, b = expert(x, *s["shared"], ws, ew)
        y, tol = y + a, tol + b
    tol = tol + 40 * U * y.abs()
    if residual:
        y = y + s["residual"].double()
        tol = tol + U * y.abs()
    return y, tol


def close(got, ref, tol):
    d = (got.double() - ref).abs()
    tol = tol + HALF[got.dtype] * (ref.abs() + tol) + TINY[got.dtype]
    assert torch.all(d <= tol), f"off by {float((d / tol).max()):.3g} tolerances, rows {torch.nonzero((d > tol).any(1)).view(-1).tolist()}"


def call(ops, s, k, norm, ws, **kw):
    return ops.moe_ffn_decode(s["x"], s["routerW"], s["gate"], s["up"], s["down"], k, norm, ws, shared=s["shared"],
                              shexp_gate=s["shexp_gate"], **kw)


CASES = [  # N, D, E, F, k, Fs, gated, norm, residual, skew
    (1, 8, 1, 8, 1, 0, False, False, False, 0), (1, 64, 2, 16, 2, 0, False, True, True, 0), (2, 264, 8, 128, 2, 0, False, False, False, 0),
    (1, 2048, 64, 1024, 8, 0, False, False, False, 0), (8, 2048, 64, 1024, 8, 0, False, False, True, 0),
    (5, 2048, 256, 512, 8, 512, True, True, False, 0), (9, 512, 16, 256, 4, 256, False, True, True, 0),
    (16, 1000, 40, 72, 6, 0, False, False, False, 1.0), (17, 256, 65, 1032, 3, 24, True, False, False, 0),
    (32, 2048, 128, 768, 8, 0, False, True, False, 1.8), (32, 128, 4, 64, 4, 64, True, False, True, 0),
    (3, 4096, 10, 96, 2, 40, False, False, False, 0), (32, 72, 1024, 8, 32, 0, False, True, False, 0),
    (7, 1024, 300, 40, 5, 0, False, False, False, 0), (31, 5000, 5, 2056, 2, 0, False, False, False, 0), (1, 8, 3, 8, 3, 8, True, True, True, 0),
    (8, 776, 24, 600, 4, 520, True, True, False, 0), (13, 640, 12, 1000, 3, 0, False, False, True, 0), (30, 904, 40, 520, 6, 72, False, True, False, 1.5),
    (4, 9000, 6, 16, 2, 0, False, False, False, 0), (8, 16, 33, 3000, 1, 0, False, True, False, 0),
    (32, 32768, 2, 16, 1, 0, False, False, False, 0), (6, 32, 2, 65536, 1, 0, False, False, True, 0), (32, 2056, 9, 24, 9, 8, False, False, False, 0),
]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("N,D,E,F,k,Fs,gated,norm,residual,skew", CASES)
def test_layer(ops, N, D, E, F, k, Fs, gated, norm, residual, skew, dtype):
    s = layer(N, D, E, F, dtype, Fs, gated, seed=1, skew=skew)
    ws = ops.new_decode_workspace(N, D, E, F, k, Fs)
    out = torch.full((N, D + 1), 7.0, dtype=dtype, device="cuda")
    call(ops, s, k, norm, ws, residual=s["residual"] if residual else None, out=out[:, :D])
    assert ops.moe_workspace_status(ws) == 0
    close(out[:, :D], *reference(s, k, norm, residual))
    assert torch.all(out[:, D] == 7)


@pytest.mark.parametrize("scale", [2.0 ** -12, 2.0 ** 9, 2.0 ** 14])
def test_intermediates_beyond_fp16(ops, scale):
    """SiLU(gate) * up beyond fp16's largest and near its smallest values, the results in its range."""
    s = layer(6, 512, 8, 128, F16, 64, True, seed=2, h_scale=1.0)
    s["up"] = s["up"] * (scale if scale < 2 ** 10 else 2.0 ** 10)
    s["x"] = s["x"] * (1.0 if scale < 2 ** 10 else 4.0)
    s["routerW"] = s["routerW"] / (1.0 if scale < 2 ** 10 else 4.0)
    s["down"] = s["down"] * 2.0 ** -6
    ws = ops.new_decode_workspace(6, 512, 8, 128, 2, 64)
    close(call(ops, s, 2, True, ws), *reference(s, 2, True))


def test_equal_logits_take_the_lower_expert(ops):
    s = layer(4, 64, 70, 16, BF16, seed=3)
    s["routerW"][:] = s["routerW"][0]
    ws = ops.new_decode_workspace(4, 64, 70, 16, 3)
    out = call(ops, s, 3, False, ws)
    x = s["x"].double()
    y, tol = torch.zeros_like(x), torch.zeros_like(x)
    w = torch.full((4,), 1 / 70, dtype=torch.float64, device="cuda")
    for e in range(3):
        a, b = expert(x, s["gate"][e], s["up"][e], s["down"][e], w, torch.full_like(w, 64 * U))
        y, tol = y + a, tol + b
    close(out, y, tol + 40 * U * y.abs())


@pytest.mark.parametrize("E", [20, 100, 600])
def test_nan_and_infinity_stay_in_their_rows(ops, E):
    s = layer(12, 256, E, 64, F16, seed=4)
    ws = ops.new_decode_workspace(12, 256, E, 64, 4)
    clean = call(ops, s, 4, True, ws)
    s["x"][2, 7], s["x"][9, 0] = float("nan"), float("inf")
    out = call(ops, s, 4, True, ws)
    keep = [i for i in range(12) if i not in (2, 9)]
    close(out[keep], *(v[keep] for v in reference_of(clean, out)))
    assert torch.all(torch.isnan(out[2])) and torch.all(torch.isnan(out[9])) and ops.moe_workspace_status(ws) == 0


def reference_of(clean, like):
    """The clean call's rows; other tokens' experts leave a row's own sums as they are but for the power of two its
    h is scaled by, which rounds nothing: equal up to one step of the type."""
    ref = clean.double()
    return ref, HALF[like.dtype] * ref.abs()


@pytest.mark.parametrize("N", [8, 9])
def test_weights_that_are_not_finite_reach_their_experts_tokens_only(ops, N):
    s = layer(N, 64, 6, 16, BF16, seed=14)
    ws = ops.new_decode_workspace(N, 64, 6, 16, 2)
    clean = call(ops, s, 2, False, ws)
    idx = torch.topk(s["x"].double() @ s["routerW"].double().t(), 2, dim=1).indices
    e = int(idx[0, 0])
    hit = (idx == e).any(dim=1)
    assert not hit.all()
    s["down"][e, :, 3] = float("inf")
    s["gate"][e, 2] = float("nan")
    out = call(ops, s, 2, False, ws)
    assert torch.equal(out[~hit], clean[~hit]) and not torch.isfinite(out[hit]).any()


def test_masked_experts(ops):
    """Experts whose logit is -inf are never chosen; a token with fewer finite logits than slots gives NaN nowhere else."""
    s = layer(5, 64, 12, 16, BF16, seed=5)
    s["x"][:, 0] = 1
    s["routerW"][3:9, 0] = float("-inf")
    ws = ops.new_decode_workspace(5, 64, 12, 16, 4)
    out = call(ops, s, 4, True, ws)
    t = dict(s)
    live = [0, 1, 2, 9, 10, 11]
    for n in ("routerW", "gate", "up", "down"):
        t[n] = s[n][live].contiguous()
    close(out, *reference(t, 4, True))


def test_strides_in_place_and_one_row_for_all(ops):
    s = layer(6, 128, 8, 64, BF16, seed=6)
    ws = ops.new_decode_workspace(6, 128, 8, 64, 2)
    plain = call(ops, s, 2, True, ws, residual=s["residual"])
    wide = torch.zeros((6, 136), dtype=BF16, device="cuda")
    wide[:, :128] = s["x"]
    stream = torch.zeros((6, 131), dtype=BF16, device="cuda")
    stream[:, :128] = s["residual"]
    t = dict(s, x=wide[:, :128])
    out = call(ops, t, 2, True, ws, residual=stream[:, :128], out=stream[:, :128])
    assert torch.equal(out, plain) and torch.all(stream[:, 128:] == 0)
    one = dict(s, x=s["x"][:1].expand(6, 128))
    y = call(ops, one, 2, True, ws)
    assert all(torch.equal(y[i], y[0]) for i in range(6))


def test_batches_share_a_workspace_and_graphs(ops):
    """Batches of other sizes on one workspace in turn, captured and replayed: the same bits each time."""
    s = layer(20, 512, 32, 96, BF16, 64, True, seed=7)
    ws = ops.new_decode_workspace(20, 512, 32, 96, 4, 64)
    parts = [dict(s, x=s["x"][:n]) for n in (20, 1, 8, 9)]
    first = [call(ops, p, 4, True, ws) for p in parts]
    graphs, outs = [], []
    for p in parts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(ops, p, 4, True, ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs)) and ops.moe_workspace_status(ws) == 0
    st = torch.cuda.Stream()
    other = ops.new_decode_workspace(20, 512, 32, 96, 4, 64)
    st.wait_stream(torch.cuda.current_stream())
    y = call(ops, parts[2], 4, True, other, stream=st)
    st.synchronize()
    assert torch.equal(y, first[2])


def test_two_calls_at_once(ops):
    """On two streams with a workspace each, among other kernels on a third: the same bits as alone."""
    a, b = layer(8, 1024, 16, 256, BF16, seed=15), layer(20, 512, 32, 96, F16, seed=16)
    wa, wb = ops.new_decode_workspace(8, 1024, 16, 256, 4), ops.new_decode_workspace(20, 512, 32, 96, 4)
    want = call(ops, a, 4, True, wa), call(ops, b, 4, True, wb)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.empty_like(want[i]) for _ in range(10)] for i in range(2)]
    busy = torch.zeros(1 << 22, device="cuda")
    torch.cuda.synchronize()
    for n in range(10):
        call(ops, a, 4, True, wa, out=outs[0][n], stream=streams[0])
        call(ops, b, 4, True, wb, out=outs[1][n], stream=streams[1])
        with torch.cuda.stream(streams[2]):
            busy.add_(1)
    torch.cuda.synchronize()
    for i, ws in enumerate((wa, wb)):
        assert ops.moe_workspace_status(ws) == 0 and all(torch.equal(o, want[i]) for o in outs[i])


def test_barrier_timeout(ops):
    """A grid barrier that cannot complete ends with MOE_DEV_TIMEOUT, out untouched, and the next call is right."""
    s = layer(3, 256, 8, 64, BF16, seed=8)
    ws = ops.new_decode_workspace(3, 256, 8, 64, 2)
    out = torch.full((3, 256), 4.0, dtype=BF16, device="cuda")
    ops.moe_debug_decode_barrier_timeout(s["x"], s["routerW"], s["gate"], s["up"], s["down"], 2, out, 50, ws)
    assert ops.moe_workspace_status(ws) == 4 and torch.all(out == 4)  # MOE_DEV_TIMEOUT
    ops.moe_workspace_init(ws)
    close(call(ops, s, 2, False, ws), *reference(s, 2, False))
    assert ops.moe_workspace_status(ws) == 0


def test_block_of_a_model(ops):
    """A pre-norm block: norm, router, and the experts' sum onto the residual, once by the whole layer's kernel and once
    by sort, products and unsort; and its norm's gradient.  Both sides round the normed rows alike; the second rounds h
    and the experts' rows to the type as well: three half steps of the sum of their magnitudes."""
    N, D, E, F, k = 24, 512, 16, 128, 4
    s = layer(N, D, E, F, BF16, seed=9)
    gamma, beta = torch.rand(D, generator=gen(10), device="cuda") + 0.5, torch.randn(D, generator=gen(11), device="cuda") * 0.1
    stream = s["residual"]
    s["x"] = ops.moe_layernorm(stream, gamma, beta, 1e-5)
    ws = ops.new_decode_workspace(N, D, E, F, k)
    out = call(ops, s, k, True, ws, residual=stream)
    close(out, *reference(s, k, True, True))

    sws = ops.new_sort_workspace(N, k, E)
    idx, w = ops.moe_topk_from_logits((s["x"].float() @ s["routerW"].t()).contiguous(), k, True)
    rows, start, tok, slot, row = ops.moe_sort_tokens(s["x"], idx, E, sws)
    h = ops.moe_matmul(rows, s["gate"], sws, expStart=start, w_up=s["up"], act="silu")
    y = ops.moe_matmul(h, s["down"], sws, expStart=start)
    got = ops.moe_unsort_tokens(y, row, w, sws).double() + stream.double()
    ref, tol = reference(s, k, True, True)
    of = torch.bucketize(torch.arange(N * k, device="cuda"), start[1:].long(), right=True)
    mag = torch.einsum("nf,ndf->nd", h.double().abs(), s["down"][of].double().abs())
    at = torch.zeros((N, D), dtype=torch.float64, device="cuda")
    at.index_add_(0, tok.long(), mag * w.double()[tok.long(), slot.long()].unsqueeze(1))
    d = (got - ref).abs()
    assert torch.all(d <= tol + 3 * HALF[BF16] * at)

    nws = ops.new_norm_workspace(N, D)
    d_y = torch.ones_like(stream)
    d_x, d_gamma, d_beta = ops.moe_layernorm_grad(d_y, stream, gamma, 1e-5, nws)
    assert d_x.shape == stream.shape and torch.equal(d_beta, torch.full((D,), float(N), device="cuda"))


def test_refusals(ops):
    s = layer(4, 64, 8, 32, BF16, 16, True, seed=12)
    ws = ops.new_decode_workspace(4, 64, 8, 32, 2, 16)
    wide = torch.zeros((4, 65), dtype=BF16, device="cuda")
    many = layer(33, 64, 8, 32, BF16, seed=13)
    for bad in (lambda: call(ops, s, 0, False, ws), lambda: call(ops, s, 9, False, ws), lambda: call(ops, many, 2, False, ws),
                lambda: call(ops, s, 2, False, ws[:256]), lambda: call(ops, dict(s, x=wide[:, 1:]), 2, False, ws),
                lambda: call(ops, s, 2, False, ws, out=s["x"]), lambda: call(ops, dict(s, shared=None), 2, False, ws),
                lambda: ops.moe_decode_workspace_size(33, 64, 8, 32, 2), lambda: ops.moe_decode_workspace_size(4, 60, 8, 32, 2)):
        with pytest.raises(ops.MoeError):
            bad()
    for bad in (lambda: call(ops, dict(s, x=s["x"].float()), 2, False, ws), lambda: call(ops, dict(s, gate=s["gate"].half()), 2, False, ws),
                lambda: call(ops, dict(s, down=s["up"]), 2, False, ws), lambda: call(ops, dict(s, routerW=s["routerW"].bfloat16()), 2, False, ws),
                lambda: call(ops, s, 2, False, ws, residual=s["residual"][:2]), lambda: call(ops, dict(s, up=s["up"].cpu()), 2, False, ws)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("N", [3, 12])
def test_a_workspace_whose_barrier_ran_out_is_refused(ops, N):
    """Its arrival count says nothing any more: calls, captured ones among them, leave out alone and say so, also after
    the status has been cleared, until the workspace is initialised."""
    s = layer(N, 256, 8, 64, BF16, seed=17)
    ws = ops.new_decode_workspace(N, 256, 8, 64, 2)
    want = call(ops, s, 2, False, ws)
    out = torch.full((N, 256), 4.0, dtype=BF16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ops, s, 2, False, ws, out=out)
    ops.moe_debug_decode_barrier_timeout(s["x"], s["routerW"], s["gate"], s["up"], s["down"], 2, out, 50, ws)
    assert ops.moe_workspace_status(ws) == 4 and torch.all(out == 4)  # MOE_DEV_TIMEOUT; read and cleared
    assert ops.moe_workspace_status(ws) == 0
    call(ops, s, 2, False, ws, out=out)
    assert ops.moe_workspace_status(ws) == 4 and torch.all(out == 4)
    g.replay()
    assert ops.moe_workspace_status(ws) == 4 and torch.all(out == 4)
    ops.moe_workspace_init(ws)
    for _ in range(3):
        g.replay()
        assert torch.equal(out, want) and torch.equal(call(ops, s, 2, False, ws), want)
    assert ops.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("N,D,E,F,k,Fs", [(2, 512, 16, 96, 3, 0), (8, 2048, 64, 1024, 8, 0), (5, 1000, 40, 1544, 4, 72), (8, 5000, 9, 2056, 2, 0),
                                          (9, 640, 24, 520, 4, 64), (32, 2048, 128, 768, 8, 0), (17, 5000, 9, 1096, 2, 1032)])
def test_a_tokens_row_does_not_hang_on_the_others(ops, N, D, E, F, k, Fs, dtype):
    """The order of a token's sums is its own: the same bits whatever the other rows hold and choose.  The residual takes
    the rounded result away, so that what is left shows the sums' last bits."""
    s = layer(N, D, E, F, dtype, Fs, Fs > 0, seed=21)
    ws = ops.new_decode_workspace(N, D, E, F, k, Fs)
    left = -call(ops, s, k, True, ws)
    want = call(ops, s, k, True, ws, residual=left)
    for i in range(6):
        keep = (5 * i) % N
        x = torch.randn((N, D), generator=gen(22 + i), device="cuda").to(dtype)
        x[keep] = s["x"][keep]
        got = call(ops, dict(s, x=x), k, True, ws, residual=left)
        assert torch.equal(got[keep], want[keep]), f"{int((got[keep] != want[keep]).sum())} of {D} values, batch {i}"


@pytest.mark.parametrize("N", [3, 20])
@pytest.mark.parametrize("apart", [2.0 ** 10, 2.0 ** 18, 2.0 ** 24])
def test_fp16_intermediates_far_apart(ops, N, apart):
    """One power of two scales all of a token's h, so its smaller values are off by 2^-39 of the largest, or 2^-22 of
    themselves (17 binades below the largest the first takes over).  The shared expert's h are the large ones; its down
    rows are 0, so that what shows is the routed experts'."""
    D, E, F, k = 256, 6, 64, 2
    s = layer(N, D, E, F, F16, F, False, seed=18)
    s["up"] = (s["up"].float() / 64).half()
    s["shared"] = ((s["shared"][0].float() * 8).half(), (s["shared"][1].float() * (apart / 64 / 8)).half(), torch.zeros_like(s["shared"][2]))
    assert torch.isfinite(s["shared"][1]).all()
    y, tol = reference(s, k, True)
    x = s["x"].double()
    a, b = x @ s["shared"][0].double().t(), x @ s["shared"][1].double().t()
    top = (a * torch.sigmoid(a) * b).abs().amax(dim=1, keepdim=True)
    rows = s["down"].double().abs().sum(dim=2).amax(dim=0)  # the largest sum of a row of down, by output
    ws = ops.new_decode_workspace(N, D, E, F, k, F)
    close(call(ops, s, k, True, ws), y, tol + 2.0 ** -39 * top * k * rows)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,dtype", [(4, BF16), (4, F16), (12, BF16), (12, F16)])
def test_tokens_with_fewer_experts_than_slots_and_with_none(ops, N, dtype, norm):
    """Logits of one token overflow to -inf for all experts but two (four slots: those two count, the others 0), of another
    for all experts (its row is NaN); the other tokens meet 0 times those weights."""
    s = layer(N, 128, 10, 64, dtype, seed=19)
    live = [2, 5]
    dead = [e for e in range(10) if e not in live]
    s["x"][:, :2] = 0
    s["x"][1, 0] = s["x"][3, 1] = -4
    s["routerW"][dead, 0] = 2e38
    s["routerW"][:, 1] = 2e38
    s["routerW"][live, 0] = 0.5
    ws = ops.new_decode_workspace(N, 128, 10, 64, 4)
    out = call(ops, s, 4, norm, ws)
    assert torch.all(torch.isnan(out[3])) and ops.moe_workspace_status(ws) == 0
    few = dict(s, x=s["x"][1:2], **{n: s[n][live].contiguous() for n in ("routerW", "gate", "up", "down")})
    close(out[1:2], *reference(few, 2, norm))
    rest = [t for t in range(N) if t not in (1, 3)]
    close(out[rest], *reference(dict(s, x=s["x"][rest]), 4, norm))


def test_gradient_of_a_blocks_norm(ops):
    """The norm before the layer and its gradient on the same residual stream, as a block runs them, d_x and d_gamma
    against float64.  fp32 sums of 512 random values: some 50 steps of 2^-24 of their magnitudes, under 2^-16 of the rows'
    scale with all factors (a gamma of 1.5, r near 1, h below 5); then half a step."""
    N, D, E, F, k = 24, 512, 16, 128, 4
    s = layer(N, D, E, F, BF16, seed=9)
    gamma, beta = torch.rand(D, generator=gen(10), device="cuda") + 0.5, torch.randn(D, generator=gen(11), device="cuda") * 0.1
    stream, d_y = s["residual"], torch.randn((N, D), generator=gen(20), device="cuda").to(BF16)
    x = ops.moe_layernorm(stream, gamma, beta, 1e-5)
    call(ops, dict(s, x=x), k, True, ops.new_decode_workspace(N, D, E, F, k), residual=stream)
    got = ops.moe_layernorm_grad(d_y, stream, gamma, 1e-5, ops.new_norm_workspace(N, D))
    leaves = [t.double().requires_grad_() for t in (stream, gamma, beta)]
    d = leaves[0] - leaves[0].mean(dim=1, keepdim=True)
    y = d / torch.sqrt(d.square().mean(dim=1, keepdim=True) + 1e-5) * leaves[1] + leaves[2]
    y.backward(d_y.double())
    for a, leaf in zip(got, leaves):
        ref = leaf.grad
        half = HALF.get(a.dtype, U)
        assert torch.all((a.double() - ref).abs() <= 2.0 ** -16 * ref.abs().amax() + half * ref.abs())
