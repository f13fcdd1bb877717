"""Token rows sorted by expert and back, the gradients of both and of the routing weights, called
through the C ABI, against plain float64 computations on the same inputs.

Tolerances, with u = 2^-24 (fp32) and h = half a step of the element type relative to the value
(2^-24, 2^-11, 2^-8):
  - rows, CSR arrays, tokRow: equal;
  - a weighted sum of k rows: k fused multiply-adds in fp32, k u sum|w r|, then one rounding, h |value|;
  - d_rows: one fp32 product, one rounding, (u + h) |value|;
  - d_topk_w: a sum of D products in fp32 in any order, D u sum|products|;
  - d_logits: see topk_grad_tolerance.
fp16 results below the normal range are multiples of 2^-24: half of that is added.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
TYPES = [torch.float32, torch.float16, torch.bfloat16]


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


def routing(N, E, k, drop, seed=0):
    g = gen(seed)
    idx = torch.topk(torch.randn((N, E), generator=g, device="cuda"), k, dim=1).indices.to(torch.int32)
    if drop:
        idx[torch.rand((N, k), generator=g, device="cuda") < drop] = -1
    return idx.contiguous()


def order(idx, E):
    """(expStart, rows' entries, tokRow) of the stable order by expert, in numpy."""
    flat = idx.cpu().numpy().reshape(-1)
    entries = np.concatenate([np.flatnonzero(flat == e) for e in range(E)])
    start = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    row = np.full(flat.size, -1, np.int64)
    row[entries] = np.arange(entries.size)
    return start, entries, row.reshape(idx.shape)


def values(shape, dtype, seed, pad=0, shift=0):
    """Random rows `pad` elements further apart than their length, their first element `shift` elements in."""
    n, d = shape
    buf = torch.randn(n * (d + pad) + shift, generator=gen(seed), device="cuda").to(dtype)
    return buf[shift:].view(n, d + pad)[:, :d] if pad or shift else buf.view(n, d)


def check_sort(ops, x, idx, E):
    N, k = idx.shape
    D = x.shape[1]
    ws = ops.new_sort_workspace(N, k, E)
    rows = torch.full((N * k, D), 7.5, dtype=x.dtype, device="cuda")
    got = ops.moe_sort_tokens(x, idx, E, ws, rows=rows)
    assert ops.moe_workspace_status(ws) == 0
    start, entries, row = order(idx, E)
    kept = entries.size
    assert np.array_equal(got[1].cpu().numpy(), start)
    tail = np.full(N * k - kept, -1)
    assert np.array_equal(got[2].cpu().numpy(), np.concatenate([entries // k, tail]))
    assert np.array_equal(got[3].cpu().numpy(), np.concatenate([entries % k, tail]))
    assert np.array_equal(got[4].cpu().numpy(), row)
    assert torch.equal(got[0][:kept], x[torch.from_numpy(entries // k).cuda()])
    assert torch.all(got[0][kept:] == 7.5)  # rows behind the last one stay as they were
    return got


SHAPES = [  # N, D, E, k, drop, pad, shift
    (1, 1, 1, 1, 0.0, 0, 0), (1, 2048, 64, 8, 0.0, 0, 0), (4, 64, 1, 1, 0.0, 0, 0), (7, 33, 5, 3, 0.3, 0, 0),
    (64, 256, 8, 2, 0.0, 0, 0), (130, 1001, 60, 6, 0.25, 0, 0), (153, 40, 1024, 32, 0.1, 0, 0),
    (300, 72, 17, 17, 0.5, 8, 0), (511, 520, 128, 8, 0.0, 1, 0), (700, 96, 33, 4, 0.9, 0, 1), (2048, 2048, 64, 8, 0.0, 0, 0),
    (1537, 136, 300, 12, 0.05, 24, 3), (5000, 16, 3, 2, 0.2, 0, 0), (97, 9000, 4, 2, 0.0, 0, 0),
    (3000, 37, 20, 3, 0.1, 0, 0), (2500, 44, 256, 2, 0.0, 2, 2),
]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,D,E,k,drop,pad,shift", SHAPES)
def test_sort(ops, N, D, E, k, drop, pad, shift, dtype):
    check_sort(ops, values((N, D), dtype, 1, pad, shift), routing(N, E, k, drop, N), E)


@pytest.mark.parametrize("N", [1, 3, 200, 4000])
def test_sort_masks_that_leave_experts_or_tokens_empty(ops, N):
    x = values((N, 24), torch.bfloat16, 2)
    check_sort(ops, x, torch.full((N, 4), -1, dtype=torch.int32, device="cuda"), 9)           # nothing kept
    check_sort(ops, x, torch.full((N, 4), 8, dtype=torch.int32, device="cuda"), 9)            # one expert, all slots
    idx = torch.full((N, 4), -1, dtype=torch.int32, device="cuda")
    idx[-1, 2] = 3
    check_sort(ops, x, idx, 9)                                                                # a single entry
    idx = torch.randint(-1, 3, (N, 4), generator=gen(3), device="cuda", dtype=torch.int32)    # experts repeated in a token
    check_sort(ops, x, idx, 9)


def test_sort_equals_bucket(ops):
    idx = routing(2048, 64, 8, 0.0)
    ws = torch.empty(max(ops.lib().moe_bucket_workspace_size(2048, 8, 64), ops.moe_sort_workspace_size(2048, 8, 64)),
                     dtype=torch.uint8, device="cuda")
    ops.moe_workspace_init(ws)
    es, ti, tk = ops.moe_bucket(idx, 64, ws)
    got = ops.moe_sort_tokens(values((2048, 8), torch.float32, 0), idx, 64, ws)
    assert torch.equal(got[1], es) and torch.equal(got[2], ti) and torch.equal(got[3], tk)


@pytest.mark.parametrize("bad", [-2, 16, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("N", [5, 3000])
def test_sort_flags_bad_experts_and_drops_them(ops, bad, N):
    idx = routing(N, 16, 2, 0.1)
    want = idx.clone()
    idx[N - 2, 1], want[N - 2, 1] = bad, -1
    x = values((N, 48), torch.float16, 0)
    ws = ops.new_sort_workspace(N, 2, 16)
    got = ops.moe_sort_tokens(x, idx, 16, ws)
    assert ops.moe_workspace_status(ws) == 1
    ref = ops.moe_sort_tokens(x, want, 16, ws)
    assert ops.moe_workspace_status(ws) == 0
    n = int(ref[1][-1])
    assert torch.equal(got[0][:n], ref[0][:n]) and all(torch.equal(a, b) for a, b in zip(got[1:], ref[1:]))


def weighted_sum(rows, row, w):
    """(sum, sum of magnitudes) in float64."""
    r = torch.from_numpy(row).cuda()
    there = (r >= 0).unsqueeze(-1)
    v = torch.where(there, rows.double()[r.clamp(min=0)] * w.double().unsqueeze(-1), 0.0)
    return v.sum(1), v.abs().sum(1)


def close(got, ref, tol):
    d = (got.double() - ref).abs()
    assert torch.all(d <= tol), f"off by {float((d / tol.clamp(min=1e-300)).max()):.3g} tolerances"


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,D,E,k,drop,pad,shift", SHAPES)
def test_unsort_and_gradients(ops, N, D, E, k, drop, pad, shift, dtype):
    idx = routing(N, E, k, drop, N)
    _, entries, row = order(idx, E)
    tokRow = torch.from_numpy(row.astype(np.int32)).cuda()
    rows = values((N * k, D), dtype, 4, 0, shift)
    rows[entries.size:] = float("nan")  # rows that no entry names
    w = torch.randn((N, k), generator=gen(5), device="cuda")
    w[tokRow < 0] = float("inf")  # a dropped entry's weight is not used
    used = torch.where(tokRow >= 0, w, 0.0)
    ws = ops.new_sort_workspace(1, 1, 1)
    wide = torch.full((N, D + pad), 3.0, dtype=dtype, device="cuda")
    out = ops.moe_unsort_tokens(rows, tokRow, w, ws, out=wide[:, :D])
    ref, mag = weighted_sum(rows, row, used)
    close(out, ref, k * U * mag + HALF[dtype] * ref.abs() * 1.001 + TINY[dtype])
    assert torch.all(wide[:, D:] == 3.0)
    d_x = ops.moe_sort_tokens_grad(rows, tokRow, ws)
    ref, mag = weighted_sum(rows, row, torch.ones_like(w))
    close(d_x, ref, k * U * mag + HALF[dtype] * ref.abs() * 1.001 + TINY[dtype])
    assert torch.all(out[torch.all(tokRow < 0, dim=1)] == 0) and torch.all(d_x[torch.all(tokRow < 0, dim=1)] == 0)

    d_out = values((N, D), dtype, 6, pad, shift)
    d_rows = torch.full((N * k, D), -2.0, dtype=dtype, device="cuda")
    d_rows, d_w = ops.moe_unsort_tokens_grad(d_out, rows, tokRow, w, ws, d_rows=d_rows)
    at = torch.from_numpy(entries).cuda()
    ref = used.double().reshape(-1)[at].unsqueeze(1) * d_out.double()[at // k]
    n = entries.size
    close(d_rows[:n], ref, (U + HALF[dtype]) * ref.abs() * 1.001 + TINY[dtype])
    assert torch.all(d_rows[n:] == -2.0)
    prod = rows.double()[:n] * d_out.double()[at // k]
    ref = torch.zeros(N * k, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    ref[at], mag[at] = prod.sum(1), prod.abs().sum(1)
    close(d_w.reshape(-1), ref, D * U * mag)
    assert ops.moe_workspace_status(ws) == 0


def test_unsort_gradient_of_one_row_for_all(ops):
    """d_out of a sum over tokens is one row, broadcast: a stride of 0 is read as it stands."""
    idx = routing(65, 8, 2, 0.2)
    _, entries, row = order(idx, 8)
    tokRow = torch.from_numpy(row.astype(np.int32)).cuda()
    rows, w = values((130, 40), torch.bfloat16, 1), torch.rand((65, 2), generator=gen(2), device="cuda")
    one = values((1, 40), torch.bfloat16, 3)
    ws = ops.new_sort_workspace(1, 1, 1)
    a = ops.moe_unsort_tokens_grad(one.expand(65, 40), rows, tokRow, w, ws)
    b = ops.moe_unsort_tokens_grad(one.repeat(65, 1), rows, tokRow, w, ws)
    assert torch.equal(a[1], b[1]) and torch.equal(a[0][:entries.size], b[0][:entries.size])
    x = one.expand(65, 40)
    assert torch.equal(ops.moe_sort_tokens(x, idx, 8, ops.new_sort_workspace(65, 2, 8))[0][:entries.size],
                       x[torch.from_numpy(entries // 2).cuda()])


def test_unsort_flags_bad_rows_and_drops_them(ops):
    rows, w = values((12, 40), torch.float32, 1), torch.rand((6, 2), generator=gen(2), device="cuda")
    row = torch.arange(12, device="cuda", dtype=torch.int32).view(6, 2)
    want = row.clone()
    ws = ops.new_sort_workspace(1, 1, 1)
    for bad in (12, -2, 2 ** 31 - 1, -2 ** 31):
        row[3, 1], want[3, 1] = bad, -1
        got = [ops.moe_unsort_tokens(rows, row, w, ws), ops.moe_sort_tokens_grad(rows, row, ws)]
        keep = torch.zeros_like(rows)
        got += ops.moe_unsort_tokens_grad(rows[:6], rows, row, w, ws, d_rows=keep)
        assert ops.moe_workspace_status(ws) == 2
        keep2 = torch.zeros_like(rows)
        ref = [ops.moe_unsort_tokens(rows, want, w, ws), ops.moe_sort_tokens_grad(rows, want, ws)]
        ref += ops.moe_unsort_tokens_grad(rows[:6], rows, want, w, ws, d_rows=keep2)
        assert ops.moe_workspace_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_unsort_equals_combine(ops):
    """fp32 rows in CSR order give moe_combine's bits for the same rows in (token, slot) order."""
    idx = routing(300, 16, 4, 0.0)
    _, entries, row = order(idx, 16)
    tokRow = torch.from_numpy(row.astype(np.int32)).cuda()
    rows, w = values((1200, 128), torch.float32, 1), torch.rand((300, 4), generator=gen(2), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    assert torch.equal(ops.moe_unsort_tokens(rows, tokRow, w, ws), ops.moe_combine(rows[tokRow.reshape(-1).long()], w))


def test_unsort_infinities_and_nan_stay_in_their_token(ops):
    rows = values((8, 16), torch.float16, 1)
    rows[2, 3], rows[5, 4] = float("nan"), float("inf")
    tokRow = torch.arange(8, device="cuda", dtype=torch.int32).view(4, 2)
    w = torch.ones((4, 2), device="cuda")
    out = ops.moe_unsort_tokens(rows, tokRow, w, ops.new_sort_workspace(1, 1, 1))
    assert torch.isnan(out[1, 3]) and out[2, 4] == float("inf")
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 3] = bad[2, 4] = True
    assert torch.all(torch.isfinite(out) | bad)


def topk_grad_reference(l, idx, d_w, norm):
    """(d_logits, tolerance) in float64, token by token over the selected experts.

    expf is within 2 ulp of its rounded argument, whose rounding moves it by |l - m| u; the sum of n terms
    adds n u, the division u: p is within (4 + L + n) u of itself, L = max |l - m|.  c = sum p v adds n u
    sum p|v|; then p (v - c) two more roundings."""
    l, d_w = l.double(), d_w.double()
    N, E = l.shape
    v = torch.zeros_like(l)
    sel = torch.zeros((N, E), dtype=torch.bool, device=l.device)
    for s in range(idx.shape[1]):
        t = torch.nonzero(idx[:, s] >= 0).squeeze(1)
        v[t, idx[t, s].long()] += d_w[t, s]
        sel[t, idx[t, s].long()] = True
    m = torch.where(sel, l, -torch.inf) if norm else l
    some = torch.any(m > -torch.inf, dim=1, keepdim=True)
    p = torch.where(some, torch.softmax(torch.where(some, m, 0.0), dim=1), 0.0)
    pv = (p * v.abs()).sum(1, keepdim=True)
    far = torch.where(torch.isfinite(m), (m - m.amax(1, keepdim=True)).abs(), 0.0).amax(1, keepdim=True)
    d = (4 + far + E) * U
    ref = p * (v - (p * v).sum(1, keepdim=True))
    return ref, (d + 3 * U) * ref.abs() + p * (d + E * U) * 2 * pv + 2.0 ** -149


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (1, 64, 8), (5, 2, 2), (33, 31, 4), (2048, 64, 8), (77, 65, 32), (300, 128, 8),
                                   (19, 257, 7), (9, 700, 16), (6, 1024, 32)])
def test_topk_grad(ops, N, E, k, norm):
    l = 3 * torch.randn((N, E), generator=gen(N), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    idx, _ = ops.moe_topk_from_logits(l, k, norm)
    d_w = torch.randn((N, k), generator=gen(E), device="cuda")
    ref, tol = topk_grad_reference(l, idx, d_w, norm)
    close(ops.moe_topk_grad(l, idx, d_w, norm, ws), ref, tol)
    # slots dropped, and an expert named twice
    idx[0, 0] = -1
    idx[-1] = idx[-1, -1].item()
    ref, tol = topk_grad_reference(l, idx, d_w, norm)
    close(ops.moe_topk_grad(l, idx, d_w, norm, ws), ref, tol)
    assert ops.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,E,k", [(77, 65, 12), (13, 200, 16), (40, 250, 17), (5003, 33, 3), (6001, 64, 8), (4999, 96, 8),
                                   (5001, 203, 7), (9999, 256, 1)])
def test_topk_grad_tokens_of_a_warp(ops, N, E, k, norm):
    """Several tokens a warp, some without anything to choose from."""
    l = 3 * torch.randn((N, E), generator=gen(N), device="cuda")
    l[::5] = -torch.inf
    l[1::7, : E // 2] = -torch.inf
    idx = torch.stack([torch.randperm(E, generator=gen(s), device="cuda")[:k] for s in range(8)]).int()
    idx = idx[torch.arange(N, device="cuda") % 8].contiguous()
    idx[2::3, 0] = -1
    ws = ops.new_sort_workspace(1, 1, 1)
    d_w = torch.randn((N, k), generator=gen(E), device="cuda")
    got = ops.moe_topk_grad(l, idx, d_w, norm, ws)
    lost = (l.gather(1, idx.clamp(min=0).long()).masked_fill(idx < 0, -torch.inf) == -torch.inf).all(1)
    none = lost if norm else (l == -torch.inf).all(1)
    assert torch.all(got[none] == 0)
    ref, tol = topk_grad_reference(l[~none], idx[~none], d_w[~none], norm)
    close(got[~none], ref, tol)
    assert ops.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("norm", [False, True])
def test_topk_grad_masked_and_extreme_logits(ops, norm):
    l = torch.randn((6, 40), generator=gen(1), device="cuda")
    l[0, 5:] = -torch.inf                      # experts masked out
    l[1] = -torch.inf                          # all of them
    l[2] = torch.finfo(torch.float32).min      # the type's lowest value throughout
    l[3] *= 1e4
    l[4, 7] = 3e38
    idx, _ = ops.moe_topk_from_logits(l, 4, norm)
    idx[1] = torch.arange(4, device="cuda", dtype=torch.int32)
    idx[5] = -1
    d_w = torch.randn((6, 4), generator=gen(2), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    got = ops.moe_topk_grad(l, idx, d_w, norm, ws)
    ref, tol = topk_grad_reference(l, idx, d_w, norm)
    assert torch.all(torch.isfinite(got)) and torch.all(got[1] == 0) and torch.all(got[5] == 0)
    close(got, ref, torch.nan_to_num(tol, posinf=0.0) + 1e-30)
    idx[0, 1] = 40
    ops.moe_topk_grad(l, idx, d_w, norm, ws)
    assert ops.moe_workspace_status(ws) == 1


@pytest.mark.parametrize("norm", [False, True])
def test_topk_grad_against_differences(ops, norm):
    """Central differences of the routing weights: h^2 / 6 times the third derivative of a softmax (at most 1
    in magnitude per weight) plus the weights' rounding, 40 u, over 2 h."""
    N, E, k, h = 7, 24, 4, 2.0 ** -6
    l = torch.randn((N, E), generator=gen(3), device="cuda")
    l[:, :k] += 6.0  # the selection stays under steps of h
    idx, _ = ops.moe_topk_from_logits(l, k, norm)
    d_w = torch.randn((N, k), generator=gen(4), device="cuda")
    got = ops.moe_topk_grad(l, idx, d_w, norm, ops.new_sort_workspace(1, 1, 1)).double()

    def loss(x):
        i, w = ops.moe_topk_from_logits(x, k, norm)
        dense = torch.zeros((N, E), dtype=torch.float64, device="cuda").scatter(1, i.long(), w.double())
        return (dense.gather(1, idx.long()) * d_w.double()).sum(1)

    tol = d_w.double().abs().sum(1) * (h * h / 6 + 40 * U / h)
    for e in range(E):
        step = torch.zeros_like(l)
        step[:, e] = h
        up, down = l + step, l - step
        d = (loss(up) - loss(down)) / (up[:, e].double() - down[:, e].double())
        assert torch.all((d - got[:, e]).abs() <= tol)


def test_unsort_gradient_against_differences(ops):
    """out is linear in rows and in the weights: a step of any size gives the derivative, up to fp32 rounding."""
    N, D, E, k = 12, 33, 5, 3
    idx = routing(N, E, k, 0.2)
    _, entries, row = order(idx, E)
    tokRow = torch.from_numpy(row.astype(np.int32)).cuda()
    rows, step = values((N * k, D), torch.float32, 1), values((N * k, D), torch.float32, 2)
    w, w_step = (torch.randn((N, k), generator=gen(s), device="cuda") for s in (3, 4))
    d_out = values((N, D), torch.float32, 5)
    ws = ops.new_sort_workspace(1, 1, 1)
    d_rows, d_w = ops.moe_unsort_tokens_grad(d_out, rows, tokRow, w, ws)

    def loss(r, x):
        return float((ops.moe_unsort_tokens(r, tokRow, x, ws).double() * d_out.double()).sum())

    scale = U * 4 * (k + D) * float(d_out.abs().double().sum()) * 40  # |rows|, |w| and the steps are below 6
    n = entries.size
    kept = tokRow >= 0
    assert abs(loss(rows + step, w) - loss(rows, w) - float((d_rows[:n].double() * step[:n].double()).sum())) <= scale
    assert abs(loss(rows, w + w_step) - loss(rows, w) - float((d_w.double() * w_step.double())[kept].sum())) <= scale


def test_training_step_of_a_layer(ops):
    """Router weights, sort, experts in torch, unsort, and the whole way back, against autograd in float64."""
    N, D, F, E, k = 96, 64, 48, 6, 2
    g = gen(11)
    x = torch.randn((N, D), generator=g, device="cuda")
    wr, w1, w2 = (torch.randn(s, generator=g, device="cuda") / 8 for s in ((E, D), (E, D, F), (E, F, D)))
    d_out = torch.randn((N, D), generator=g, device="cuda")
    ws = ops.new_sort_workspace(N, k, E)
    logits = (x.double() @ wr.double().t()).float()
    idx, w = ops.moe_topk_from_logits(logits, k, True)
    rows, start, _, _, tokRow = ops.moe_sort_tokens(x, idx, E, ws)
    seg = start.tolist()
    h, y = torch.empty((N * k, F), device="cuda", dtype=torch.float64), torch.empty_like(rows)
    for e in range(E):
        s = slice(seg[e], seg[e + 1])
        h[s] = torch.relu(rows[s].double() @ w1[e].double())
        y[s] = (h[s] @ w2[e].double()).float()
    out = ops.moe_unsort_tokens(y, tokRow, w, ws)
    d_y, d_w = ops.moe_unsort_tokens_grad(d_out, y, tokRow, w, ws)
    d_in = torch.empty_like(rows)
    for e in range(E):
        s = slice(seg[e], seg[e + 1])
        d_in[s] = (((d_y[s].double() @ w2[e].double().t()) * (h[s] > 0)) @ w1[e].double().t()).float()
    d_x = ops.moe_sort_tokens_grad(d_in, tokRow, ws)
    d_l = ops.moe_topk_grad(logits, idx, d_w, True, ws)
    assert ops.moe_workspace_status(ws) == 0

    X = x.double().requires_grad_()
    L = (X.detach() @ wr.double().t()).float().double().requires_grad_()
    p = torch.softmax(L, 1)
    sel = p.gather(1, idx.long())
    W = sel / sel.sum(1, keepdim=True)
    O = 0
    for s in range(k):
        e = idx[:, s].long()
        O = O + W[:, s:s + 1] * (torch.relu((X.unsqueeze(1) @ w1.double()[e])) @ w2.double()[e]).squeeze(1)
    O.backward(d_out.double())
    # fp32 roundings of O(1) values through sums of at most 64 terms of size below 40
    for got, ref in ((out, O.detach()), (d_x, X.grad), (d_l, L.grad)):
        assert float((got.double() - ref).abs().max()) <= 64 * 40 * U * max(1.0, float(ref.abs().max()))


def test_replayed_graph_and_side_stream(ops):
    """Captured calls on new inputs give what plain calls give, and a call follows the stream it is given."""
    N, D, E, k = 300, 200, 12, 3
    x, idx, w = values((N, D), torch.bfloat16, 1), routing(N, E, k, 0.1), torch.rand((N, k), generator=gen(2), device="cuda")
    ws = ops.new_sort_workspace(N, k, E)
    rows = torch.zeros((N * k, D), dtype=torch.bfloat16, device="cuda")

    def step():
        r, _, _, _, row = ops.moe_sort_tokens(x, idx, E, ws, rows=rows)
        out = ops.moe_unsort_tokens(r, row, w, ws)
        d_rows, d_w = ops.moe_unsort_tokens_grad(out, r, row, w, ws, d_rows=torch.zeros_like(r))
        return out, d_rows, d_w, ops.moe_sort_tokens_grad(d_rows, row, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (5, 6):
        x.copy_(values((N, D), torch.bfloat16, seed))
        idx.copy_(routing(N, E, k, 0.2, seed))
        rows.zero_()
        graph.replay()
        got = [t.clone() for t in captured]
        rows.zero_()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    side = torch.cuda.Stream()
    big = torch.randn((4096, 4096), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-3
        x.copy_(values((N, D), torch.bfloat16, 9))
        got = ops.moe_sort_tokens(x, idx, E, ws)[0]
    side.synchronize()
    n = int((idx >= 0).sum())
    assert torch.equal(got[:n], ops.moe_sort_tokens(x, idx, E, ws)[0][:n])


def test_two_threads_at_once(ops):
    """Calls from two host threads, each on a stream and with a workspace of its own."""
    import threading

    got = {}

    def work(seed):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ws = ops.new_sort_workspace(3000, 4, 400)
            for i in range(10):
                E = (400, 12)[i % 2]
                idx = routing(3000, E, 4, 0.1, seed + i)
                x = values((3000, 64 + 8 * i), torch.bfloat16, seed)
                rows, start, tok, _, row = ops.moe_sort_tokens(x, idx, E, ws)
                w = torch.ones((3000, 4), device="cuda")
                out = ops.moe_unsort_tokens(rows, row, w, ws)
                kept = (idx >= 0).sum(1, keepdim=True)
                got[seed, i] = bool(torch.equal(out, (x.float() * kept).bfloat16())) and int(start[-1]) == int(kept.sum())

    threads = [threading.Thread(target=work, args=(s,)) for s in (100, 200)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 20 and all(got.values())


def test_stream_argument(ops):
    """Work and outputs follow the stream that is passed, whatever the current one is."""
    x, idx = values((900, 72), torch.float16, 1), routing(900, 20, 4, 0.1)
    ws = ops.new_sort_workspace(900, 4, 20)
    want = ops.moe_sort_tokens(x, idx, 20, ws)
    n = int(want[1][-1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.moe_sort_tokens(x, idx, 20, ws, stream=side)
    w = torch.rand((900, 4), generator=gen(2), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    out = ops.moe_unsort_tokens(got[0], got[4], w, ws, stream=side)
    d_rows, d_w = ops.moe_unsort_tokens_grad(out, got[0], got[4], w, ws, stream=side)
    d_x = ops.moe_sort_tokens_grad(got[0], got[4], ws, stream=side)
    side.synchronize()
    assert torch.equal(got[0][:n], want[0][:n]) and all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert torch.equal(out, ops.moe_unsort_tokens(want[0], want[4], w, ws))
    assert torch.equal(d_w, ops.moe_unsort_tokens_grad(out, want[0], want[4], w, ws)[1])
    assert torch.equal(d_x, ops.moe_sort_tokens_grad(want[0], want[4], ws))


def test_rows_past_32_bit_offsets(ops):
    N, D, E, k = 40000, 7000, 8, 8  # 2.24e9 elements in the sorted rows
    idx = torch.randint(0, 3, (N, k), generator=gen(1), device="cuda", dtype=torch.int32)
    x = values((N, D), torch.bfloat16, 1)
    ws = ops.new_sort_workspace(N, k, E)
    rows, _, tok, _, row = ops.moe_sort_tokens(x, idx, E, ws)
    for r in (0, 1, N * k // 2, 2 ** 31 // D - 1, 2 ** 31 // D, 2 ** 31 // D + 1, N * k - 1):
        assert torch.equal(rows[r], x[int(tok[r])])
    w = torch.ones((N, k), device="cuda")
    out = ops.moe_unsort_tokens(rows, row, w, ws)
    assert torch.equal(out, x * 8)  # eight equal rows: exact
    d_rows, d_w = ops.moe_unsort_tokens_grad(x, rows, row, w, ws)
    assert torch.equal(d_rows, rows)
    t = torch.arange(0, N, 997, device="cuda")
    ref = (x[t].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    close(d_w[t], ref, D * U * ref)
    assert ops.moe_workspace_status(ws) == 0


def test_refused_tensors(ops):
    x, idx = values((6, 16), torch.float32, 1), routing(6, 4, 2, 0.0)
    ws = ops.new_sort_workspace(6, 2, 4)
    rows, _, _, _, row = ops.moe_sort_tokens(x, idx, 4, ws)
    w = torch.rand((6, 2), device="cuda")
    for call in (lambda: ops.moe_sort_tokens(x.t(), idx[:2], 4, ws),                       # rows not contiguous
                 lambda: ops.moe_sort_tokens(x.double(), idx, 4, ws),                      # type
                 lambda: ops.moe_sort_tokens(x, idx.long(), 4, ws),
                 lambda: ops.moe_sort_tokens(x, idx[:5], 4, ws),                           # shape
                 lambda: ops.moe_sort_tokens(x, idx, 4, ws, rows=rows[:11]),
                 lambda: ops.moe_unsort_tokens(rows, row, w.double(), ws),
                 lambda: ops.moe_unsort_tokens(rows, row, w[:, :1], ws),
                 lambda: ops.moe_unsort_tokens(rows, row, w, ws, out=x.half()),
                 lambda: ops.moe_unsort_tokens_grad(x.half(), rows, row, w, ws),
                 lambda: ops.moe_sort_tokens(x.cpu(), idx, 4, ws),                         # device
                 lambda: ops.moe_sort_tokens(x, idx.cpu(), 4, ws)):
        with pytest.raises(ValueError):
            call()
    buf = torch.zeros((12, 16), device="cuda")
    for call, code in ((lambda: ops.moe_sort_tokens(buf[:6], idx, 4, ws, rows=buf), -1),   # output over input
                       (lambda: ops.moe_unsort_tokens(buf, row, w, ws, out=buf[6:]), -1),
                       (lambda: ops.moe_unsort_tokens_grad(x, buf, row, w, ws, d_rows=buf), -1),
                       (lambda: ops.moe_unsort_tokens(rows, row, w, ws, out=x[:1].expand(6, 16)), -1),
                       (lambda: ops.moe_sort_tokens(x, idx, 4, ws[:256]), -3),
                       (lambda: ops.moe_sort_tokens(x, idx, 4, ws[1:]), -1),               # misaligned workspace
                       (lambda: ops.moe_sort_tokens(x, idx, 1, ws), -2),                   # top_k > E
                       (lambda: ops.moe_sort_tokens(x, idx, 1025, ws), -2),
                       (lambda: ops.moe_sort_tokens(x[:0], idx[:0], 4, ws), -1)):
        with pytest.raises(ops.MoeError) as err:
            call()
        assert err.value.code == code
    assert ops.moe_workspace_status(ws) == 0


def test_sort_of_a_routing_that_lies_in_the_workspace(ops):
    """A layer's workspace serves the sort of the routing that the layer left in it: only the scratch at its start may
    not hold arguments."""
    from mixture_experts_ffn_top_gb300.workloads import WORKLOADS, make_inputs

    wl = WORKLOADS["tiny"]
    inp = make_inputs(wl)
    layer = ops.MoeLayer.from_numpy(inp, device="cuda:0", top_k=wl.top_k, max_tokens=wl.N)
    x = torch.from_numpy(np.ascontiguousarray(inp["hidden"])).cuda()
    layer.prefill(x, wl.top_k, wl.norm_topk_prob)
    views = ops.moe_workspace_views(layer.ws, wl.N, wl.D, wl.E, wl.F, wl.top_k, layer.w.Fs)
    idx, weights, start = (views[n].clone() for n in ("topk_idx", "topk_w", "expStart"))
    got = ops.moe_sort_tokens(x, views["topk_idx"], wl.E, layer.ws)
    ref = ops.moe_sort_tokens(x, idx, wl.E, ops.new_sort_workspace(wl.N, wl.top_k, wl.E))
    assert all(torch.equal(a, b) for a, b in zip(got, ref)) and torch.equal(got[1], start)
    assert torch.equal(views["topk_idx"], idx) and torch.equal(views["topk_w"], weights)
    assert layer.status() == 0
    inside = layer.ws[256:256 + 4 * idx.numel()].view(torch.int32).view(wl.N, wl.top_k)
    with pytest.raises(ops.MoeError) as err:
        ops.moe_sort_tokens(x, inside, wl.E, layer.ws)
    assert err.value.code == -1


@pytest.mark.parametrize("N,D,E,k", [(3, 64, 8, 2), (700, 2048, 16, 4), (2048, 9000, 300, 3)])
def test_sort_gives_up_copies_that_never_complete(ops, N, D, E, k):
    """Every warp's first wait runs out, then its waits for the other copies in flight: a timeout in the status word
    within bounds, the order as ever, no row written, and the same workspace serves the next call."""
    import time

    x, idx = values((N, D), torch.bfloat16, 1), routing(N, E, k, 0.1)
    ws = ops.new_sort_workspace(N, k, E)
    rows = torch.full((N * k, D), 7.5, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    since = time.time()
    got = ops.moe_debug_sort_wait_timeout(x, idx, E, rows, 20, ws)
    assert ops.moe_workspace_status(ws) == 4  # synchronises
    assert time.time() - since < 10  # five waits of 20 ms a CTA, every CTA in one wave
    assert torch.all(rows == 7.5)
    ref = ops.moe_sort_tokens(x, idx, E, ws, rows=rows)
    assert ops.moe_workspace_status(ws) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, ref[1:]))
    _, entries, _ = order(idx, E)
    assert torch.equal(rows[:entries.size], x[torch.from_numpy(entries // k).cuda()])


def test_sort_wait_check_needs_bulk_copies(ops):
    idx = routing(6, 4, 2, 0.0)
    rows, ws = torch.zeros((12, 33), dtype=torch.bfloat16, device="cuda"), ops.new_sort_workspace(6, 2, 4)
    for x, out, ms, code in ((values((6, 33), torch.bfloat16, 1), rows, 20, -2),
                             (values((6, 32), torch.bfloat16, 1), rows[:, :32].contiguous(), 0, -1)):
        with pytest.raises(ops.MoeError) as err:
            ops.moe_debug_sort_wait_timeout(x, idx, 4, out, ms, ws)
        assert err.value.code == code


@pytest.mark.parametrize("N,D,E,k,drop,pad,shift,dtype", [
    (40000, 24, 64, 8, 0.3, 0, 0, torch.bfloat16), (40000, 25, 64, 8, 0.1, 3, 1, torch.float16),
    (20001, 16, 1024, 17, 0.6, 8, 0, torch.float32), (320001, 9, 3, 1, 0.2, 0, 0, torch.float32),
    (11000, 8, 300, 32, 0.95, 0, 0, torch.float16), (38912, 33, 40, 8, 0.0, 0, 0, torch.bfloat16)])
def test_sort_of_ranges_whose_ranks_wait_in_the_output(ops, N, D, E, k, drop, pad, shift, dtype):
    """More than 2048 entries a range: their ranks wait in tokRow itself, for bulk copies and plain ones, with dropped
    entries, whole tokens without any, and experts out of range among them.  (38912 x 8 is exactly 2048 a range.)"""
    idx = routing(N, E, k, drop, N)
    idx[N // 2: N // 2 + 300] = -1
    x = values((N, D), dtype, 1, pad, shift)
    check_sort(ops, x, idx, E)
    want = idx.clone()
    idx[::1009, 0], want[::1009, 0] = E, -1
    ws = ops.new_sort_workspace(N, k, E)
    got = ops.moe_sort_tokens(x, idx, E, ws)
    assert ops.moe_workspace_status(ws) == 1
    ref = ops.moe_sort_tokens(x, want, E, ws)
    n = int(ref[1][-1])
    assert torch.equal(got[0][:n], ref[0][:n]) and all(torch.equal(a, b) for a, b in zip(got[1:], ref[1:]))


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,E,k", [(8, 40, 4), (9, 257, 7), (5000, 64, 8), (5003, 129, 3)])
def test_topk_grad_of_far_apart_logits(ops, norm, N, E, k):
    """Logits thousands and 3e38 apart, to the accuracy of near ones.  As topk_grad_reference, with L = max |l - m| taken
    over the experts whose probability is not 0 in fp32 alone (expf is 0 below -104, exactly): those at 0 add nothing to
    any sum, and where they stand for a probability below 2^-149 that and its gradient are off by less than 2^-146."""
    l = torch.randn((N, E), generator=gen(N), device="cuda")
    l[0::8] *= 1e4
    l[1::8, 7] = 3e38
    l[2::8] = torch.finfo(torch.float32).min
    l[2::8, 3] = -3e38
    l[3::8] *= 30
    l[4::8, E // 2:] = -torch.inf
    l[5::8, 1::2] -= 103.0  # on the edge of what expf returns
    idx, _ = ops.moe_topk_from_logits(l, k, norm)
    d_w = torch.randn((N, k), generator=gen(E), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    got = ops.moe_topk_grad(l, idx, d_w, norm, ws)
    assert ops.moe_workspace_status(ws) == 0
    L, v = l.double(), torch.zeros((N, E), dtype=torch.float64, device="cuda")
    v.scatter_(1, idx.long(), d_w.double())
    chosen = torch.zeros((N, E), dtype=torch.bool, device="cuda").scatter_(1, idx.long(), True)
    m = torch.where(chosen, L, -torch.inf) if norm else L
    p = torch.softmax(m, dim=1)
    below = m.amax(1, keepdim=True) - m
    far = torch.where(below < 104, below, 0.0).amax(1, keepdim=True)
    ref = p * (v - (p * v).sum(1, keepdim=True))
    d, pv = (4 + far + E) * U, (p * v.abs()).sum(1, keepdim=True)
    close(got, ref, (d + 3 * U) * ref.abs() + p * (d + E * U) * 2 * pv + 2.0 ** -146 * (v.abs() + pv + 1))
    assert torch.all(got[1::8].abs() <= 2.0 ** -146)  # one expert has it all: nothing moves


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,E,k", [(16, 64, 8), (5000, 64, 8), (5003, 203, 7), (40, 700, 20)])
def test_topk_grad_nan_and_infinity_stay_in_their_token(ops, norm, N, E, k):
    l = torch.randn((N, E), generator=gen(N), device="cuda")
    idx, _ = ops.moe_topk_from_logits(l, k, norm)
    d_w = torch.randn((N, k), generator=gen(E), device="cuda")
    ws = ops.new_sort_workspace(1, 1, 1)
    clean = ops.moe_topk_grad(l, idx, d_w, norm, ws)
    t = torch.arange(N, device="cuda")
    l[t[3::9], idx[3::9, 0].long()] = float("nan")
    l[t[5::9], idx[5::9, k - 1].long()] = float("inf")
    d_w[7::9, 1] = float("nan")
    got = ops.moe_topk_grad(l, idx, d_w, norm, ws)
    bad = (t % 9 == 3) | (t % 9 == 5) | (t % 9 == 7)
    assert torch.equal(got[~bad], clean[~bad])
    assert torch.all(torch.isnan(got[bad].gather(1, idx[bad].long())))  # as the formula: every selected expert's
    if norm:
        others = torch.ones_like(got, dtype=torch.bool).scatter_(1, idx.long(), False)
        assert torch.all(got[others] == 0)
    else:
        assert torch.all(torch.isnan(got[bad]))
