"""What is measured of the operators around the routed experts.

  sort         token rows sorted by expert (and the CSR of that order); its gradient
  unsort       sorted rows back to their tokens, weighted by the routing weights; its gradient
  topk_grad    the gradient of the routing weights down to the router's logits
  w4           products with 4-bit weights and group scales: one matrix, or one per expert over
               sorted rows; plain, or gate and up with SwiGLU

``run`` computes the plain form in elementary torch operations, or with ``own`` set makes the calls
of the framework.
"""
import math

import numpy as np
import torch

own = False

_ops = None


def _framework():
    global _ops
    if _ops is None:
        from mixture_experts_ffn_top_gb300 import ops

        _ops = ops
    return _ops


DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
BYTES = {"float32": 4, "float16": 2, "bfloat16": 2}


def _tokens(name, op, N, D, E, k, dtype, grad=False, drop=0.0, skew=0.0, pad=0):
    return {"name": name, "op": op, "grad": grad, "N": N, "D": D, "E": E, "k": k, "dtype": dtype, "drop": drop,
            "skew": skew, "pad": pad}


def _w4(name, E, k, tokens, R, K, group, dtype, zeros=False, pair=False):
    return {"name": name, "op": "w4", "E": E, "k": k, "N": tokens, "R": R, "K": K, "group": group, "dtype": dtype,
            "zeros": zeros, "pair": pair}


def listed():
    return [
        # a decode step of four sequences: latency
        _tokens("sort decode", "sort", 4, 2048, 64, 8, "bfloat16"),
        # the prompt batch of the default benchmark layer
        _tokens("sort prompt", "sort", 2048, 2048, 64, 8, "bfloat16"),
        # the backward of a skewed batch in fp32, the framework's own hidden type
        _tokens("sort gradient skewed", "sort", 4096, 2048, 128, 8, "float32", grad=True, skew=1.2),
        # a padded batch at an odd width: padding tokens and dropped entries leave rows empty
        _tokens("unsort ragged padded", "unsort", 517, 1001, 60, 6, "float16", drop=0.25),
        # a large training batch, forward
        _tokens("unsort training", "unsort", 8192, 2048, 64, 8, "bfloat16"),
        # the same step's backward at the benchmark layer's batch
        _tokens("unsort gradient", "unsort", 2048, 2048, 64, 8, "bfloat16", grad=True),
        # router backward of the benchmark layer
        {"name": "topk gradient", "op": "topk_grad", "N": 2048, "E": 64, "k": 8, "norm": False},
        # router backward of a long batch over many experts, weights renormalised
        {"name": "topk gradient many experts", "op": "topk_grad", "N": 16384, "E": 256, "k": 8, "norm": True},
        # one token through one square projection beside the layer: latency
        _w4("w4 one token", 1, 1, 1, 2048, 2048, 128, "bfloat16"),
        # gate/up of a decode step of eight sequences over the benchmark layer's experts
        _w4("w4 experts gate up", 64, 8, 8, 1024, 2048, 32, "float16", pair=True),
        # down of 32 sequences in fp32 with zero points, at a narrow expert width
        _w4("w4 experts down", 128, 8, 32, 2048, 768, 64, "float32", zeros=True),
        # an output head for eight sequences: the weights' stream alone
        _w4("w4 head", 1, 1, 8, 131072, 4096, 128, "float16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "sort", "unsort", "unsort", "topk_grad", "w4", "w4", "w4"])
    dtype = rng.choice(sorted(DTYPES))
    if op == "topk_grad":
        E = _log(rng, 4, 512)
        return {"op": op, "N": _log(rng, 1, 16384 * 256 // max(E, 256)), "E": E, "k": rng.randint(1, min(E, 16)),
                "norm": rng.random() < 0.5}
    if op == "w4":
        E = 1 if rng.random() < 0.4 else _log(rng, 2, 128)
        group = rng.choice([32, 64, 128])
        K = group * max(1, _log(rng, 128, 8192) // group)
        pair = rng.random() < 0.4
        k = 1 if E == 1 else rng.randint(1, min(E, 8))
        N = _log(rng, 1, 48)
        # the plain form of the experts holds a matrix for each row: at most 2 GB
        top = 131072 * 4096 // (K * E * (1 + pair)) if E == 1 else min(131072 * 4096 // (K * E), 2 ** 28 // (N * k * K)) // (1 + pair)
        c = _w4("", E, k, N, max(1, _log(rng, 32, max(33, min(top, 65536)))), K, group, dtype, rng.random() < 0.4, pair)
        del c["name"]
        return c
    D = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        D = D // 8 * 8
    E = _log(rng, 2, 512)
    k = rng.randint(1, min(E, 12))
    grad = rng.random() < 0.5
    most = 8192 * 8 * 2048 // (D * k * (BYTES[dtype] // 2) * (2 if grad else 1))
    c = _tokens("", op, _log(rng, 1, max(2, min(most, 16384))), D, E, k, dtype, grad,
                rng.choice([0.0, 0.0, 0.1, 0.5]), rng.choice([0.0, 1.2]), rng.choice([0, 0, 8, 40]))
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --
def _routing(g, N, E, k, skew, drop):
    """topk_idx [N][k] int32: the k largest of random logits, some experts ahead of the others where
    skewed; with drops every eighth token is padding and single entries are dropped."""
    logits = torch.randn((N, E), generator=g, device="cuda")
    if skew:
        rank = torch.randperm(E, generator=g, device="cuda").float()
        logits = logits - 1.5 * skew * torch.log(rank + 1)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    if drop:
        gone = torch.rand((N, k), generator=g, device="cuda") < drop
        gone |= torch.rand((N, 1), generator=g, device="cuda") < 0.125
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
    return idx.contiguous()


def _order(idx, E):
    """Entries by (expert, token, slot), dropped ones last: the entry of each row, each entry's row, offsets."""
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    by, entry = torch.sort(key, stable=True)
    start = torch.searchsorted(by, torch.arange(E + 1, device=by.device)).to(torch.int32)
    row = torch.empty_like(entry)
    row[entry] = torch.arange(entry.numel(), device=entry.device)
    row = torch.where(flat < 0, torch.full_like(row, -1), row)
    return entry, by < E, row.reshape(idx.shape).to(torch.int32), start


def _strided(t, pad):
    """The same values in rows that lie `pad` values further apart, as in a slice of a wider buffer."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, N, E, k = case["op"], case["N"], case["E"], case["k"]
    s = {"case": case}
    if op == "topk_grad":
        s["logits"] = torch.randn((N, E), generator=g, device="cuda")
        s["idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        s["d_w"] = torch.randn((N, k), generator=g, device="cuda")
        if own:
            s["ws"] = _framework().new_sort_workspace(N, k, E)
        return s
    dtype = DTYPES[case["dtype"]]
    if op == "w4":
        R, K, G = case["R"], case["K"], case["group"]
        n = N * k
        s["start"] = None if E == 1 else _order(_routing(g, N, E, k, 0.0, 0.0), E)[3]
        s["x"] = torch.randn((n, K), generator=g, device="cuda").to(dtype)
        mats = []
        for _ in range(2 if case["pair"] else 1):
            q = torch.randint(0, 256, (E, R, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            sc = (torch.rand((E, R, K // G), generator=g, device="cuda") + 0.5) * (0.2 / math.sqrt(K))
            sc = sc.to(torch.bfloat16 if dtype == torch.bfloat16 else torch.float16)
            z = torch.randint(0, 16, (E, R, K // G), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
            mats.append((q, sc, z))
        s["mats"] = mats
        if own:  # the weights' handle and the status words, kept by a program as long as the weights
            s["w"] = _framework().MoeW4Weights(*mats[0], *(mats[1] if case["pair"] else ()))
            s["ws"] = _framework().new_sort_workspace(1, 1, 1)
        return s
    D = case["D"]
    s["idx"] = _routing(g, N, E, k, case["skew"], case["drop"])
    _, _, s["row"], _ = _order(s["idx"], E)
    if op == "sort" and not case["grad"]:
        s["x"] = _strided(torch.randn((N, D), generator=g, device="cuda").to(dtype), case["pad"])
        s["rows"] = torch.zeros((N * k, D), dtype=dtype, device="cuda")
    else:
        s["rows"] = torch.randn((N * k, D), generator=g, device="cuda").to(dtype)
        w = torch.rand((N, k), generator=g, device="cuda") + 0.05
        s["w"] = w / w.sum(dim=1, keepdim=True)
        if op == "unsort" and case["grad"]:
            s["d_out"] = _strided(torch.randn((N, D), generator=g, device="cuda").to(dtype), case["pad"])
            s["d_rows"] = torch.zeros((N * k, D), dtype=dtype, device="cuda")
    if own:
        s["ws"] = _framework().new_sort_workspace(N, k, E)
    return s


# -------------------------------------------------------------------- run --
def _codes(q):
    return torch.stack((q & 15, q >> 4), dim=-1).reshape(*q.shape[:-1], q.shape[-1] * 2)


def _weights(q, sc, z, G):
    """[E][R][K] fp32 of packed codes (even columns in the low nibbles), scales and zero points."""
    v = _codes(q).float().reshape(*sc.shape, G)
    v = v - (8.0 if z is None else z.float().unsqueeze(-1))
    return (v * sc.float().unsqueeze(-1)).reshape(*q.shape[:-1], q.shape[-1] * 2)


def _expert_of(start, n):
    return torch.searchsorted(start.long(), torch.arange(n, device=start.device), right=True) - 1


def _plain_w4(s):
    c, x = s["case"], s["x"].float()
    each = []
    of = None if s["start"] is None else _expert_of(s["start"], x.shape[0])
    for q, sc, z in s["mats"]:
        if of is None:
            each.append(x @ _weights(q[0], sc[0], None if z is None else z[0], c["group"]).t())
        else:
            W = _weights(q[of], sc[of], None if z is None else z[of], c["group"])
            each.append((W @ x.unsqueeze(-1)).squeeze(-1))
    y = each[0] if len(each) == 1 else each[0] / (1 + torch.exp(-each[0])) * each[1]
    return y.to(s["x"].dtype)


def _plain_tokens(s):
    c = s["case"]
    N, k, D, E = c["N"], c["k"], c["D"], c["E"]
    if c["op"] == "sort" and not c["grad"]:
        entry, kept, row, start = _order(s["idx"], E)
        rows = torch.where(kept.unsqueeze(1), s["x"][entry // k], torch.zeros((), dtype=s["x"].dtype, device="cuda"))
        none = torch.full_like(entry, -1)
        return {"rows": rows, "expStart": start, "expTokI": torch.where(kept, entry // k, none).to(torch.int32),
                "expTokK": torch.where(kept, entry % k, none).to(torch.int32), "tokRow": row}
    row = s["row"].long()
    there = (row >= 0).unsqueeze(-1)
    dtype = s["rows"].dtype
    got = torch.where(there, s["rows"][row.clamp(min=0)].float(), torch.zeros((), device="cuda"))
    if c["op"] == "sort":
        return {"d_x": got.sum(dim=1).to(dtype)}
    if not c["grad"]:
        return {"out": (got * s["w"].unsqueeze(-1)).sum(dim=1).to(dtype)}
    d_out = s["d_out"].float().unsqueeze(1)
    d_w = (got * d_out).sum(dim=-1)
    d_rows = torch.zeros((N * k + 1, D), dtype=dtype, device="cuda")
    d_rows[torch.where(row < 0, torch.full_like(row, N * k), row)] = (s["w"].unsqueeze(-1) * d_out).to(dtype)
    return {"d_rows": d_rows[:N * k], "d_w": d_w}


def _plain_topk_grad(s):
    idx, l, d_w = s["idx"].long(), s["logits"], s["d_w"]
    if s["case"]["norm"]:
        sel = l.gather(1, idx)
        w = torch.exp(sel - sel.amax(dim=1, keepdim=True))
        w = w / w.sum(dim=1, keepdim=True)
        return {"d_logits": torch.zeros_like(l).scatter(1, idx, w * (d_w - (w * d_w).sum(dim=1, keepdim=True)))}
    p = torch.exp(l - l.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    d_p = torch.zeros_like(l).scatter(1, idx, d_w)
    return {"d_logits": p * (d_p - (p * d_p).sum(dim=1, keepdim=True))}


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return _plain_topk_grad(state) if op == "topk_grad" else {"y": _plain_w4(state)} if op == "w4" else _plain_tokens(state)
    ops, ws = _ops, state["ws"]
    if op == "topk_grad":
        return {"d_logits": ops.moe_topk_grad(state["logits"], state["idx"], state["d_w"], c["norm"], ws)}
    if op == "w4":
        return {"y": ops.moe_w4_matvec(state["w"], state["x"], state["start"], ws)}
    if op == "sort" and not c["grad"]:
        rows, start, tok, slot, row = ops.moe_sort_tokens(state["x"], state["idx"], c["E"], ws, rows=state["rows"])
        return {"rows": rows, "expStart": start, "expTokI": tok, "expTokK": slot, "tokRow": row}
    if op == "sort":
        return {"d_x": ops.moe_sort_tokens_grad(state["rows"], state["row"], ws)}
    if not c["grad"]:
        return {"out": ops.moe_unsort_tokens(state["rows"], state["row"], state["w"], ws)}
    d_rows, d_w = ops.moe_unsort_tokens_grad(state["d_out"], state["rows"], state["row"], state["w"], ws, d_rows=state["d_rows"])
    return {"d_rows": d_rows, "d_w": d_w}


# ------------------------------------------------------------------- work --
def work(case):
    op, N, E, k = case["op"], case["N"], case["E"], case["k"]
    if op == "topk_grad":
        return {"bytes": 8 * N * E + 8 * N * k, "flops": 6 * N * E}
    b = BYTES[case["dtype"]]
    if op == "w4":
        R, K, n, m = case["R"], case["K"], N * k, 2 if case["pair"] else 1
        touched = 1 if E == 1 else E * (1 - (1 - k / E) ** N)
        per = R * K / 2 + R * (K // case["group"]) * (3 if case["zeros"] else 2)
        return {"bytes": touched * m * per + n * K * b + n * R * b, "flops": 2 * n * R * K * m}
    D = case["D"]
    kept = N * k * ((1 - case["drop"]) * 0.875 if case["drop"] else 1)
    one = {"bytes": N * D * b + kept * D * b + N * k * 4, "flops": 0}
    if op == "sort" and not case["grad"]:
        return {"bytes": one["bytes"] + N * k * 12 + 4 * E, "flops": 0}
    if op == "sort":
        return {"bytes": one["bytes"], "flops": kept * D}
    if not case["grad"]:
        return {"bytes": one["bytes"] + N * k * 4, "flops": 2 * kept * D}
    return {"bytes": one["bytes"] + kept * D * b + N * k * 8, "flops": 3 * kept * D}


# ------------------------------------------------------------------ exact --
def _exact_topk_grad(s):
    """By the chain rule through the probabilities: w = p_sel (over their sum), p = softmax(l)."""
    l = s["logits"].cpu().numpy().astype(np.float64)
    idx, d_w = s["idx"].cpu().numpy(), s["d_w"].cpu().numpy().astype(np.float64)
    at = np.arange(l.shape[0])[:, None]
    p = np.exp(l - l.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    d_sel = d_w
    if s["case"]["norm"]:
        sel = p[at, idx]
        total = sel.sum(axis=1, keepdims=True)
        d_sel = d_w / total - (d_w * sel).sum(axis=1, keepdims=True) / total ** 2
    d_p = np.zeros_like(p)
    d_p[at, idx] = d_sel
    return {"d_logits": p * d_p - p * (p * d_p).sum(axis=1, keepdims=True)}


def _exact_w4(s):
    """Expert by expert: each group's integer codes against the row, less the zero point's share."""
    c = s["case"]
    x = s["x"].double()
    n, K, G = x.shape[0], c["K"], c["group"]
    J = K // G
    start = [0, n] if s["start"] is None else s["start"].tolist()
    each = [torch.zeros((n, c["R"]), dtype=torch.float64, device="cuda") for _ in s["mats"]]
    for e in range(c["E"]):
        a, b = start[e], start[e + 1]
        if a == b:
            continue
        xe = x[a:b].reshape(b - a, J, G).transpose(0, 1)  # [J][n][G]
        total = xe.sum(dim=2, keepdim=True)
        for y, (q, sc, z) in zip(each, s["mats"]):
            for lo in range(0, c["R"], 4096):
                hi = min(lo + 4096, c["R"])
                pairs = q[e, lo:hi].reshape(hi - lo, J, G // 2).transpose(0, 1)  # [J][R][G/2]
                dot = xe[:, :, 0::2] @ (pairs & 15).double().transpose(1, 2)
                dot += xe[:, :, 1::2] @ (pairs >> 4).double().transpose(1, 2)
                zero = 8.0 if z is None else z[e, lo:hi].double().t().unsqueeze(1)
                y[a:b, lo:hi] = ((dot - zero * total) * sc[e, lo:hi].double().t().unsqueeze(1)).sum(dim=0)
    if len(each) == 1:
        return {"y": each[0]}
    return {"y": each[0] * torch.sigmoid(each[0]) * each[1]}


def _exact_tokens(s):
    """Slot by slot, from the definition: entry (t, s) of expert e sits behind all entries of lower
    experts and the earlier ones of its own."""
    c = s["case"]
    N, k, D, E = c["N"], c["k"], c["D"], c["E"]
    if c["op"] == "sort" and not c["grad"]:
        idx = s["idx"].cpu().numpy().reshape(-1)
        lists = [np.flatnonzero(idx == e) for e in range(E)]
        entry = torch.from_numpy(np.concatenate(lists)).cuda()
        rows = torch.zeros((N * k, D), dtype=torch.float64, device="cuda")
        rows[:entry.numel()] = s["x"].double()[entry // k]
        return {"rows": rows, "expStart": None, "expTokI": None, "expTokK": None, "tokRow": None}
    row = s["row"].long()
    total = torch.zeros((N, D), dtype=torch.float64, device="cuda")
    d_rows = torch.zeros((N * k, D), dtype=torch.float64, device="cuda")
    d_w = torch.zeros((N, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(row[:, j] >= 0).squeeze(1)
        r = row[t, j]
        w = s["w"][t, j].double().unsqueeze(1)
        mine = s["rows"][r].double()
        if c["op"] == "sort":
            total[t] += mine
        elif not c["grad"]:
            total[t] += w * mine
        else:
            d = s["d_out"][t].double()
            d_rows[r] = w * d
            d_w[t, j] = (d * mine).sum(dim=1)
    if c["op"] == "sort":
        return {"d_x": total}
    return {"d_rows": d_rows, "d_w": d_w} if c["grad"] else {"out": total}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_topk_grad(s) if case["op"] == "topk_grad" else _exact_w4(s) if case["op"] == "w4" else _exact_tokens(s)
