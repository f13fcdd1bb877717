"""Host-side argument checks of the norms, the 16-bit products and the layer for decode batches: every refusal is
answered before any launch (no GPU here; the pointers below are never dereferenced)."""
import ctypes

import pytest

INVALID, SHAPE, SMALL = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_ffn_top_gb300 import build, ops

    build.build()
    return ops.lib()


def with_(args, **new):
    return list({**args, **new}.values())


NORM = dict(x=0x100000, xs=64, dtype=2, gamma=0x200000, beta=0x210000, eps=1e-5, N=16, D=64, y=0x300000, ys=64, stream=None)
GRAD = dict(dy=0x100000, dys=64, x=0x140000, xs=64, dtype=2, gamma=0x200000, eps=1e-5, N=16, D=64, dx=0x300000, dxs=64,
            dg=0x400000, db=0x410000, ws=0x500000, ws_bytes=1 << 20, stream=None)
RMS = {k: v for k, v in GRAD.items() if k != "db"}
MATMUL = dict(x=0x1000000, xs=64, dtype=2, w=0x2000000, up=None, bias=None, bias_up=None, act=0, res=None, rs=0, start=0x3000000,
              E=4, n=48, R=32, K=64, y=0x4000000, ys=32, ws=0x5000000, ws_bytes=256, stream=None)
DECODE = dict(x=0x1000000, xs=64, dtype=2, router=0x1100000, sg=None, gate=0x2000000, up=0x2100000, down=0x2200000, shg=None,
              shu=None, shd=None, res=None, rs=0, N=4, D=64, E=8, F=32, Fs=0, k=2, norm=1, out=0x3000000, os=64, ws=0x5000000,
              ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("name,args,nulls,outs", [
    ("moe_layernorm", NORM, ["x", "gamma", "y"], ["y"]),
    ("moe_layernorm_grad", GRAD, ["dy", "x", "gamma", "dx", "dg", "ws"], ["dx", "dg", "db"]),
    ("moe_rmsnorm_grad", RMS, ["dy", "x", "gamma", "dx", "dg", "ws"], ["dx", "dg"]),
])
def test_norms(lib, name, args, nulls, outs):
    f = getattr(lib, name)
    for n in nulls:
        assert f(*with_(args, **{n: None})) == INVALID, n
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(dtype=3), dict(dtype=-1), dict(xs=-1)):
        assert f(*with_(args, **bad)) == INVALID, bad
    for bad in (dict(N=0), dict(N=1 << 30), dict(D=0), dict(xs=(1 << 30) + 1)):
        assert f(*with_(args, **bad)) == SHAPE, bad
    wide = {n: 1 << 20 for n in ("xs", "dys", "ys", "dxs") if n in args}
    assert f(*with_(args, D=32769, **wide)) == SHAPE
    out_stride = "ys" if "ys" in args else "dxs"
    assert f(*with_(args, **{out_stride: 63})) == INVALID
    for o in outs:
        for other in [n for n in ("x", "dy", "gamma", "ws", "dx", "dg") if n in args and n != o]:
            assert f(*with_(args, **{o: args[other]})) == INVALID, (o, other)
        assert f(*with_(args, **{o: args[o] + 1})) == INVALID, o
    if "ws" in args:
        need = lib.moe_norm_workspace_size(16, 64)
        assert need >= 256 + 16 * 64 * 8 and f(*with_(args, ws_bytes=need - 1)) == SMALL and f(*with_(args, ws=0x500010)) == INVALID
    assert lib.moe_norm_workspace_size(0, 64) == 0 and lib.moe_norm_workspace_size(4, 32769) == 0


def test_matmul(lib):
    f = lib.moe_matmul
    for n in ("x", "w", "y", "ws", "start"):
        assert f(*with_(MATMUL, **{n: None})) == INVALID, n
    for bad in (dict(dtype=0), dict(dtype=3), dict(act=-1), dict(act=4), dict(bias_up=0x6000000), dict(n=0), dict(xs=63), dict(xs=0),
                dict(ys=31), dict(res=0x7000000, rs=-1), dict(x=0x1000008), dict(w=0x2000002), dict(up=0x6000008), dict(xs=68),
                dict(y=0x4000001), dict(bias=0x6000002), dict(ws=0x5000080)):
        assert f(*with_(MATMUL, **bad)) == INVALID, bad
    for bad in (dict(E=0), dict(E=1025), dict(R=0), dict(K=0), dict(K=60), dict(n=1 << 30), dict(E=1024, R=1 << 21, ys=1 << 21), dict(E=1, R=0x7fffff01, ys=1 << 31),
                dict(xs=(1 << 30) + 8)):
        assert f(*with_(MATMUL, **bad)) == SHAPE, bad
    assert f(*with_(MATMUL, ws_bytes=255)) == SMALL
    for n in ("x", "w", "start", "ws"):
        assert f(*with_(MATMUL, y=MATMUL[n])) == INVALID, n
    assert f(*with_(MATMUL, up=0x6000000, y=0x6000000)) == INVALID
    assert f(*with_(MATMUL, res=MATMUL["y"] + 64, rs=32)) == INVALID      # over y, but not y itself
    assert f(*with_(MATMUL, res=MATMUL["y"], rs=64)) == INVALID


def test_decode(lib):
    f = lib.moe_ffn_decode
    for n in ("x", "router", "gate", "up", "down", "out", "ws"):
        assert f(*with_(DECODE, **{n: None})) == INVALID, n
    shared = dict(Fs=16, shg=0x2300000, shu=0x2400000, shd=0x2500000)
    for bad in (dict(dtype=0), dict(xs=-8), dict(xs=68), dict(os=63), dict(x=0x1000008), dict(gate=0x2000008), dict(router=0x1100004),
                dict(Fs=16), dict(shg=0x2300000), {**shared, "shd": None}, {**shared, "sg": 0x2600004}, dict(sg=0x2600000),
                dict(res=0x4000001, rs=64), dict(ws=0x5000080)):
        assert f(*with_(DECODE, **bad)) == INVALID, bad
    for bad in (dict(N=0), dict(N=33), dict(k=0), dict(k=9), dict(E=0), dict(E=1025), dict(D=60), dict(F=36), dict(F=0), dict(F=65544),
                {**shared, "Fs": 12}):
        assert f(*with_(DECODE, **bad)) in (SHAPE, INVALID), bad
    need = lib.moe_decode_workspace_size(4, 64, 8, 32, 2, 0)
    assert need > 256 and f(*with_(DECODE, ws_bytes=need - 1)) == SMALL
    assert lib.moe_decode_workspace_size(4, 64, 8, 32, 2, 16) > need
    for bad in ((0, 64, 8, 32, 2, 0), (33, 64, 8, 32, 2, 0), (4, 60, 8, 32, 2, 0), (4, 64, 8, 32, 9, 0), (4, 64, 8, 30, 2, 0), (4, 64, 1025, 32, 2, 0)):
        assert lib.moe_decode_workspace_size(*bad) == 0, bad
    for n in ("x", "router", "gate", "down", "ws"):
        assert f(*with_(DECODE, out=DECODE[n])) == INVALID, n
    assert f(*with_(DECODE, res=DECODE["out"] + 2, rs=64)) == INVALID
    for ms in (0, 1001):
        assert lib.moe_debug_decode_barrier_timeout(0x1000000, 64, 2, 0x1100000, 0x2000000, 0x2100000, 0x2200000, 4, 64, 8, 32, 2,
                                                    0x3000000, 64, ms, 0x5000000, 1 << 20, None) == INVALID


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    from mixture_experts_ffn_top_gb300 import ops

    x, ws = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros(4096, dtype=torch.uint8)
    gamma, w = torch.ones(64), torch.zeros((2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.moe_layernorm(x, gamma, None, 1e-5)
    with pytest.raises(ValueError):
        ops.moe_layernorm_grad(x, x, gamma, 1e-5, ws)
    with pytest.raises(ValueError):
        ops.moe_matmul(x, w, ws)
    with pytest.raises(ValueError):
        ops.moe_ffn_decode(x, torch.zeros((2, 64)), w, w, w.transpose(1, 2), 1, False, ws)
