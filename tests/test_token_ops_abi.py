"""Host-side argument checks of the token sort, its gradients and the 4-bit products: every refusal is
answered before any CUDA call (no GPU here; the pointers below are never dereferenced)."""
import ctypes

import pytest

V, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
INVALID, SHAPE, SMALL = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_ffn_top_gb300 import build, ops

    build.build()
    return ops.lib()


def with_(args, **new):
    return list({**args, **new}.values())


SORT = dict(x=0x100000, x_stride=64, dtype=2, idx=0x200000, N=16, k=2, E=8, D=64, start=0x300000, tok=0x310000,
            slot=0x320000, row=0x330000, rows=0x400000, ws=0x500000, ws_bytes=1 << 16, stream=None)
SORT_GRAD = dict(d_rows=0x100000, n=32, dtype=0, row=0x200000, N=16, k=2, D=64, d_x=0x300000, stride=64, ws=0x500000,
                 ws_bytes=256, stream=None)
UNSORT = dict(rows=0x100000, n=32, dtype=0, row=0x200000, w=0x210000, N=16, k=2, D=64, out=0x300000, stride=64,
              ws=0x500000, ws_bytes=256, stream=None)
UNSORT_GRAD = dict(d_out=0x100000, stride=64, rows=0x200000, n=32, dtype=1, row=0x300000, w=0x310000, N=16, k=2, D=64,
                   d_rows=0x400000, d_w=0x480000, ws=0x500000, ws_bytes=256, stream=None)
TOPK_GRAD = dict(logits=0x100000, idx=0x200000, d_w=0x210000, N=16, E=8, k=2, norm=0, d_l=0x300000, ws=0x500000,
                 ws_bytes=256, stream=None)
CREATE = dict(out=None, E=2, R=16, K=128, group=64, sdtype=1, q=0x100000, s=0x200000, z=0x300000, uq=None, us=None,
              uz=None, stream=None)


@pytest.mark.parametrize("name,args,nulls", [
    ("moe_sort_tokens", SORT, ["x", "idx", "start", "tok", "slot", "row", "rows", "ws"]),
    ("moe_sort_tokens_grad", SORT_GRAD, ["d_rows", "row", "d_x", "ws"]),
    ("moe_unsort_tokens", UNSORT, ["rows", "row", "w", "out", "ws"]),
    ("moe_unsort_tokens_grad", UNSORT_GRAD, ["d_out", "rows", "row", "w", "d_rows", "d_w", "ws"]),
    ("moe_topk_grad", TOPK_GRAD, ["logits", "idx", "d_w", "d_l", "ws"]),
])
def test_null_shape_workspace_and_overlap(lib, name, args, nulls):
    f = getattr(lib, name)
    for n in nulls:
        assert f(*with_(args, **{n: None})) == INVALID, n
    for k in (0, 33):
        assert f(*with_(args, k=k)) == SHAPE
    assert f(*with_(args, N=0)) == SHAPE and f(*with_(args, N=1 << 30)) == SHAPE
    if "E" in args:
        assert f(*with_(args, E=0)) == SHAPE and f(*with_(args, E=1025)) == SHAPE and f(*with_(args, E=1)) == SHAPE
    if "D" in args:
        assert f(*with_(args, D=0)) in (SHAPE, INVALID) and f(*with_(args, D=(1 << 24) + 1)) in (SHAPE, INVALID)
        assert f(*with_(args, dtype=3)) == INVALID and f(*with_(args, dtype=-1)) == INVALID
    if "n" in args:
        assert f(*with_(args, n=0)) == INVALID and f(*with_(args, n=1 << 30)) == SHAPE
    assert f(*with_(args, ws=0x500010)) == INVALID                # not 256-byte aligned
    assert f(*with_(args, ws_bytes=255)) == SMALL
    outs = {"moe_sort_tokens": ["start", "tok", "slot", "row", "rows"], "moe_sort_tokens_grad": ["d_x"],
            "moe_unsort_tokens": ["out"], "moe_unsort_tokens_grad": ["d_rows", "d_w"], "moe_topk_grad": ["d_l"]}[name]
    pointers = [n for n in nulls if n not in outs]
    for o in outs:                                               # an output over an input, the workspace or an output
        for other in pointers + [p for p in outs if p != o]:
            assert f(*with_(args, **{o: args[other]})) == INVALID, (o, other)
        assert f(*with_(args, **{o: args[o] + 1})) == INVALID, o   # misaligned


def test_strides(lib):
    assert lib.moe_sort_tokens(*with_(SORT, x_stride=-1)) == INVALID
    assert lib.moe_sort_tokens(*with_(SORT, x_stride=(1 << 30) + 1)) == SHAPE
    assert lib.moe_sort_tokens_grad(*with_(SORT_GRAD, stride=63)) == INVALID
    assert lib.moe_unsort_tokens(*with_(UNSORT, stride=0)) == INVALID
    assert lib.moe_unsort_tokens_grad(*with_(UNSORT_GRAD, stride=-64)) == INVALID


def test_sort_workspace_size(lib):
    f = lib.moe_sort_workspace_size
    assert f(1, 1, 1) >= 256 and f(2048, 8, 64) >= 256 + 4 * 64
    assert f(2048, 8, 1024) >= f(2048, 8, 64) >= f(8, 8, 64)
    assert f(0, 8, 64) == 0 and f(16, 33, 64) == 0 and f(16, 8, 4) == 0 and f(16, 2, 1025) == 0 and f(1 << 28, 8, 64) == 0
    assert lib.moe_sort_tokens(*with_(SORT, ws_bytes=f(16, 2, 8) - 1)) == SMALL


def test_w4_create(lib):
    h = V()
    ok = {**CREATE, "out": ctypes.byref(h)}
    assert lib.moe_w4_weights_create(*with_(ok, out=None)) == INVALID
    for n in ("q", "s"):
        assert lib.moe_w4_weights_create(*with_(ok, **{n: None})) == INVALID
    for sd in (0, 3, -1):
        assert lib.moe_w4_weights_create(*with_(ok, sdtype=sd)) == INVALID
    assert lib.moe_w4_weights_create(*with_(ok, uq=0x400000)) == INVALID                       # up without its scales
    assert lib.moe_w4_weights_create(*with_(ok, uq=0x400000, us=0x500000)) == INVALID          # and without zero points
    assert lib.moe_w4_weights_create(*with_(ok, z=None, uq=0x400000, us=0x500000, uz=0x600000)) == INVALID
    assert lib.moe_w4_weights_create(*with_(ok, uz=0x600000)) == INVALID
    assert lib.moe_w4_weights_create(*with_(ok, s=0x200001)) == INVALID
    for bad in (dict(group=16), dict(group=48), dict(group=256), dict(K=96), dict(K=0), dict(K=32896), dict(E=0),
                dict(E=1025), dict(R=0), dict(R=(1 << 24) + 1)):
        assert lib.moe_w4_weights_create(*with_(ok, **bad)) == SHAPE, bad
    assert not h.value
    assert lib.moe_w4_weights_destroy(None) == INVALID
    assert lib.moe_w4_weights_shape(None, None, None, None, None, None) == INVALID
    assert lib.moe_w4_weights_device_bytes(None) == 0
    assert lib.moe_w4_matvec(None, 0x1000, 128, 0, 0x2000, 4, 0x3000, 16, 0x4000, 256, None) == INVALID


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    from mixture_experts_ffn_top_gb300 import ops

    x, idx, w = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    for call in (lambda: ops.moe_sort_tokens(x, idx, 4, ws), lambda: ops.moe_sort_tokens_grad(x, idx, ws),
                 lambda: ops.moe_unsort_tokens(x, idx, w, ws), lambda: ops.moe_unsort_tokens_grad(x, x, idx, w, ws),
                 lambda: ops.moe_topk_grad(x, idx, w, False, ws),
                 lambda: ops.MoeW4Weights(torch.zeros((4, 16), dtype=torch.uint8), torch.ones((4, 1)).half())):
        with pytest.raises(ValueError):
            call()


def test_sort_wait_check_refuses_limits(lib):
    args = with_(SORT)
    for ms in (0, -1, 2001):
        assert lib.moe_debug_sort_wait_timeout(*args[:13], ms, *args[13:]) == INVALID
    assert lib.moe_debug_sort_wait_timeout(*with_(SORT, N=0)[:13], 20, *args[13:]) == SHAPE
    assert lib.moe_debug_sort_wait_timeout(*with_(SORT, D=63, x_stride=63)[:13], 20, *args[13:]) == SHAPE
