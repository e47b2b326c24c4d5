"""CPU tests of the operators around a block's products: what their entry points refuse, with the documented status
codes and before anything touches a GPU (pointers are made-up aligned addresses), which GPU the torch-facing calls run
on, and the 64-bit definitions' gradients against differences."""
import warnings

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp8_block_scaled_amd as gfg
from fp8_block_scaled_amd import layers, serving
from oracle import layers_oracle as lo

EINVAL, EUNSUPPORTED = 1, 2
P = 1 << 20


def lib():
    return gfg.load_library()


def last():
    return lib().grouped_fp8_last_error().decode()


# ------------------------------------------------------------------ refusals
GEMM = dict(a=P, sa=P, ld=4, b=P, sb=P, bias=None, d=P, M=4, N=5, K=64, out=0)
SIZES = [
    (dict(out=2), EINVAL), (dict(out=-1), EINVAL), (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL),
    (dict(K=40), EUNSUPPORTED), (dict(K=(1 << 22) + 16), EUNSUPPORTED), (dict(N=(1 << 28) + 1), EUNSUPPORTED),
    (dict(M=128 * 65535 + 1), EUNSUPPORTED), (dict(M=1 << 62), EUNSUPPORTED), (dict(M=1 << 21, ld=1 << 21, K=1 << 22, bytes=1 << 60), EUNSUPPORTED),
    (dict(a=None), EINVAL), (dict(b=None), EINVAL), (dict(sb=None), EINVAL), (dict(d=None), EINVAL), (dict(a=P + 8), EINVAL),
    (dict(b=P + 1), EINVAL), (dict(bias=P + 2), EINVAL), (dict(d=P + 4), EINVAL),
]


@pytest.mark.parametrize("change,code", SIZES + [(dict(sa=None), EINVAL), (dict(ld=3), EINVAL), (dict(ld=-4), EINVAL)])
def test_product_refuses(change, code):
    a = {**GEMM, **change}
    assert lib().fp8_gemm(a["a"], a["sa"], a["ld"], a["b"], a["sb"], a["bias"], a["d"], a["M"], a["N"], a["K"], a["out"], None) == code
    assert "fp8_gemm" in last()


@pytest.mark.parametrize("change,code", SIZES + [
    (dict(dt=3), EINVAL), (dict(dt=-1), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 8), EINVAL), (dict(bytes=4 * 64 + 3), EINVAL),
])
def test_linear_refuses(change, code):
    a = {**GEMM, "dt": 1, "ws": P, "bytes": 4 * 64 + 4, **change}
    assert lib().fp8_linear(a["a"], a["dt"], a["b"], a["sb"], a["bias"], a["d"], a["M"], a["N"], a["K"], a["out"], a["ws"],
                            a["bytes"], None) == code
    assert "fp8_linear" in last()


BACK = dict(dy=P, x=P, dt=1, bt=P, bts=P, dx=P, dw=P, db=P, M=4, N=32, K=64, dxt=0, dwt=0, acc=0, ws=P, bytes=1 << 40)


@pytest.mark.parametrize("change,code", [
    (dict(dt=3), EINVAL), (dict(dxt=2), EINVAL), (dict(dwt=3), EINVAL), (dict(acc=1), EINVAL), (dict(acc=1, dwt=1), EINVAL), (dict(M=-1), EINVAL),
    (dict(N=0), EINVAL), (dict(K=0), EINVAL), (dict(N=24), EUNSUPPORTED), (dict(K=24), EUNSUPPORTED), (dict(N=(1 << 22) + 16), EUNSUPPORTED),
    (dict(M=(1 << 22) + 1), EUNSUPPORTED), (dict(M=1 << 22, N=1 << 20), EUNSUPPORTED), (dict(dx=None, dw=None, db=None), EINVAL),
    (dict(dy=None), EINVAL), (dict(x=None), EINVAL), (dict(bt=None), EINVAL), (dict(bts=None), EINVAL), (dict(dy=P + 8), EINVAL),
    (dict(x=P + 8), EINVAL), (dict(bt=P + 8), EINVAL), (dict(dx=P + 4), EINVAL), (dict(dw=P + 4), EINVAL), (dict(db=P + 2), EINVAL),
    (dict(ws=None), EINVAL), (dict(ws=P + 8), EINVAL), (dict(bytes=100), EINVAL),
])
def test_backward_refuses(change, code):
    a = {**BACK, **change}
    assert lib().fp8_linear_backward(*(a[n] for n in ("dy", "x", "dt", "bt", "bts", "dx", "dw", "db", "M", "N", "K", "dxt", "dwt", "acc", "ws",
                                                     "bytes")), None) == code
    assert "fp8_linear_backward" in last()


QUANT = dict(w=P, dt=0, G=1, N=32, K=64, q=P, s=P, qt=P, st=P)


@pytest.mark.parametrize("change,code", [
    (dict(dt=3), EINVAL), (dict(G=0), EINVAL), (dict(G=65536), EINVAL), (dict(N=0), EINVAL), (dict(K=-16), EINVAL), (dict(K=24), EUNSUPPORTED),
    (dict(N=33), EUNSUPPORTED), (dict(G=65535, N=1 << 12, K=1 << 12), EUNSUPPORTED), (dict(w=None), EINVAL), (dict(q=None), EINVAL),
    (dict(s=None), EINVAL), (dict(qt=None), EINVAL), (dict(st=None), EINVAL), (dict(w=P + 8), EINVAL), (dict(q=P + 8), EINVAL),
    (dict(qt=P + 8), EINVAL),
])
def test_weight_quantizer_refuses(change, code):
    a = {**QUANT, **change}
    assert lib().fp8_quantize_weight_device(*(a[n] for n in ("w", "dt", "G", "N", "K", "q", "s", "qt", "st")), None) == code
    assert "fp8_quantize_weight_device" in last()


NORM = dict(y=P, r=P, w=P, post=P, gate=P, kind=1, alpha=1.0, eps=1e-6, out=P, z=P, stats=P, M=3, H=32, dt=1, rdt=1, q=P, s=P, ld=3)
NORM_BAD = [
    (dict(dt=3), EINVAL), (dict(dt=1, rdt=2), EINVAL), (dict(dt=0, rdt=1), EINVAL), (dict(kind=3), EINVAL), (dict(kind=0), EINVAL),
    (dict(gate=None), EINVAL), (dict(M=-1), EINVAL), (dict(H=0), EINVAL), (dict(H=32784), EUNSUPPORTED), (dict(H=7), EUNSUPPORTED), (dict(M=1 << 31), EUNSUPPORTED),
    (dict(r=None), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(y=P + 1), EINVAL), (dict(r=P + 1), EINVAL),
    (dict(out=P + 1), EINVAL), (dict(rdt=0, r=P + 2), EINVAL), (dict(w=P + 2), EINVAL), (dict(post=P + 2), EINVAL), (dict(gate=P + 1), EINVAL),
    (dict(stats=P + 2), EINVAL), (dict(w=None), EINVAL),
]


@pytest.mark.parametrize("change,code", NORM_BAD + [(dict(z=None), EINVAL), (dict(z=None, w=None, out=None), EINVAL), (dict(z=P + 1), EINVAL)])
def test_norm_refuses(change, code):
    a = {**NORM, **change}
    assert lib().residual_norm(*(a[n] for n in ("y", "r", "w", "post", "gate", "kind", "alpha", "eps", "out", "z", "stats", "M", "H", "dt", "rdt")),
                               None) == code
    assert "residual_norm" in last()


@pytest.mark.parametrize("change,code", NORM_BAD + [(dict(q=None), EINVAL), (dict(s=None), EINVAL), (dict(ld=2), EINVAL), (dict(q=P + 4), EINVAL),
                                                    (dict(H=40), EUNSUPPORTED)])
def test_norm_fp8_refuses(change, code):
    a = {**NORM, **change}
    assert lib().residual_norm_fp8(*(a[n] for n in ("y", "r", "w", "post", "gate", "kind", "alpha", "eps", "out", "q", "s", "ld", "stats", "M", "H",
                                                   "dt", "rdt")), None) == code
    assert "residual_norm_fp8" in last()


NBACK = dict(dout=P, dz=P, out=P, y=P, stats=P, w=P, post=P, gate=P, kind=1, alpha=1.0, dr=P, dy=P, dw=P, dp=P, dg=P, acc=0, M=3, H=32, dt=1, rdt=1,
             ws=P, bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(dt=3), EINVAL), (dict(rdt=2), EINVAL), (dict(kind=5), EINVAL), (dict(kind=0, gate=None), EINVAL), (dict(gate=None), EINVAL),
    (dict(H=0), EINVAL), (dict(H=40000), EUNSUPPORTED), (dict(M=1 << 31), EUNSUPPORTED), (dict(dout=None, dz=None), EINVAL), (dict(y=None), EINVAL),
    (dict(out=None), EINVAL), (dict(w=None), EINVAL), (dict(post=None), EINVAL), (dict(stats=None), EINVAL),
    (dict(dr=None, dy=None, dw=None, dp=None, dg=None), EINVAL), (dict(dout=P + 1), EINVAL), (dict(dz=P + 1), EINVAL), (dict(dy=P + 1), EINVAL),
    (dict(dw=P + 2), EINVAL), (dict(dp=P + 2), EINVAL), (dict(dg=P + 2), EINVAL), (dict(ws=None), EINVAL), (dict(ws=P + 4), EINVAL),
    (dict(bytes=3 * 2 * 32 * 4 - 1 - 4 * 32 * 4), EINVAL),
])
def test_norm_backward_refuses(change, code):
    a = {**NBACK, **change}
    assert lib().residual_norm_backward(*(a[n] for n in ("dout", "dz", "out", "y", "stats", "w", "post", "gate", "kind", "alpha", "dr", "dy", "dw", "dp",
                                                        "dg", "acc", "M", "H", "dt", "rdt", "ws", "bytes")), None) == code
    assert "residual_norm_backward" in last()


ROUTER = dict(l=P, dt=0, ids=P, off=None, loss=P, counts=P, f=P, T=3, E=8, k=2, S=1, score=0, ws=P, bytes=1 << 30, dw=P, dloss=P, dl=P)
ROUTER_BAD = [
    (dict(dt=7), EINVAL), (dict(score=2), EINVAL), (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(k=0), EINVAL), (dict(S=0), EINVAL), (dict(S=2), EINVAL),
    (dict(E=1025), EUNSUPPORTED), (dict(k=65), EUNSUPPORTED), (dict(T=1 << 31), EUNSUPPORTED), (dict(S=65536, off=P), EUNSUPPORTED),
    (dict(l=None), EINVAL), (dict(ids=None), EINVAL), (dict(l=P + 2), EINVAL), (dict(ids=P + 2), EINVAL), (dict(off=P + 1), EINVAL), (dict(f=P + 1), EINVAL),
]


@pytest.mark.parametrize("change,code", ROUTER_BAD + [
    (dict(loss=None), EINVAL), (dict(counts=None), EINVAL), (dict(f=None), EINVAL), (dict(counts=P + 2), EINVAL), (dict(loss=P + 2), EINVAL),
    (dict(ws=None), EINVAL), (dict(ws=P + 8), EINVAL), (dict(bytes=100), EINVAL)])
def test_balance_refuses(change, code):
    a = {**ROUTER, **change}
    assert lib().moe_balance_loss(*(a[n] for n in ("l", "dt", "ids", "off", "loss", "counts", "f", "T", "E", "k", "S", "score")), 0.1, 0.0, a["ws"],
                                  a["bytes"], None) == code
    assert "moe_balance_loss" in last()


@pytest.mark.parametrize("change,code", ROUTER_BAD + [(dict(dl=None), EINVAL), (dict(f=None), EINVAL), (dict(dloss=None), EINVAL),
                                                      (dict(dl=P + 2), EINVAL), (dict(dw=P + 2), EINVAL), (dict(dw=None, f=None, dloss=None), EINVAL)])
def test_router_backward_refuses(change, code):
    a = {**ROUTER, **change}
    assert lib().moe_router_backward(*(a[n] for n in ("l", "dt", "ids", "dw", "f", "dloss", "off", "dl", "T", "E", "k", "S", "score")), 1, 1.0, None) == code
    assert "moe_router_backward" in last()


def test_nothing_to_do_is_no_error():
    """No rows and nothing to sum over them: success without a launch, whatever the pointers."""
    n = None
    assert lib().fp8_gemm(n, n, 0, n, n, n, n, 0, 5, 64, 0, n) == 0
    assert lib().fp8_linear(n, 1, n, n, n, n, 0, 5, 64, 0, n, 0, n) == 0
    assert lib().fp8_linear_backward(n, n, 1, n, n, P, n, n, 0, 32, 64, 0, 0, 0, n, 0, n) == 0
    assert lib().fp8_linear_backward(n, n, 1, n, n, P, P, P, 0, 32, 64, 0, 2, 1, n, 0, n) == 0
    assert lib().residual_norm(n, n, n, n, n, 0, 1.0, 1e-6, n, n, n, 0, 32, 1, 1, n) == 0
    assert lib().residual_norm_fp8(n, n, n, n, n, 0, 1.0, 1e-6, n, n, n, 0, n, 0, 32, 1, 1, n) == 0
    assert lib().residual_norm_backward(n, n, n, n, n, n, n, n, 0, 1.0, P, n, P, n, n, 1, 0, 32, 1, 1, n, 0, n) == 0
    assert lib().moe_router_backward(n, 0, n, P, n, n, n, n, 0, 8, 2, 1, 0, 1, 1.0, n) == 0


def test_workspace_sizes():
    assert gfg.fp8_linear_workspace_bytes(7, 272) == 7 * 272 + 3 * 8 and gfg.fp8_linear_workspace_bytes(0, 64) == 0
    M, N, K = 130, 48, 272      # dy by rows, dy and x by columns (256 tokens), scales in rows of a multiple of 4, the parts of dbias
    want = M * N + 132 + N * 256 + 2 * 48 + K * 256 + 2 * 272 + 2 * N * 4
    assert want <= gfg.fp8_linear_backward_workspace_bytes(M, N, K) <= want + 7 * 15
    assert gfg.residual_norm_backward_workspace_bytes(0, 32) == 0 < gfg.residual_norm_backward_workspace_bytes(1, 32)
    assert gfg.moe_balance_workspace_bytes(0, 8, 1) >= 16


# ------------------------------------------------------------------ the binding
def test_bindings_refuse_what_is_not_on_a_gpu():
    z, bf, u8, i32 = torch.zeros, torch.bfloat16, torch.uint8, torch.int32
    for call in (
        lambda: gfg.fp8_quantize_weight_device(z(16, 16)),
        lambda: gfg.fp8_gemm(z(2, 16, dtype=u8), z(1, 2, dtype=u8), z(4, 16, dtype=u8), z(1, 1, dtype=u8), z(2, 4, dtype=bf)),
        lambda: gfg.fp8_linear(z(2, 16), z(4, 16, dtype=u8), z(1, 1, dtype=u8), z(2, 4, dtype=bf)),
        lambda: gfg.fp8_linear_backward(z(2, 16), z(2, 16), None, None, dw=z(16, 16)),
        lambda: gfg.residual_norm(z(2, 16), z(2, 16), z(16)),
        lambda: gfg.residual_norm_fp8(z(2, 16), z(2, 16), z(16)),
        lambda: gfg.residual_norm_backward(z(2, 16), None, None, z(2, 16), None, None, dresidual=z(2, 16)),
        lambda: gfg.moe_balance_loss(z(2, 8), z(2, 2, dtype=i32)),
        lambda: gfg.moe_router_backward(z(2, 8), z(2, 2, dtype=i32), z(2, 8), dweights=z(2, 2)),
    ):
        with pytest.raises(ValueError, match="must be on a GPU"):
            call()


class Library:
    """Every entry point returns 0 and notes (its name, the current device, the last argument: the stream)."""

    def __init__(self, now):
        self.now, self.seen = now, []

    def __getattr__(self, name):
        def entry(*args):
            if not name.endswith("workspace_bytes"):
                self.seen.append((name, self.now["device"], args[-1]))
            return 0
        return entry


@pytest.fixture
def world(monkeypatch):
    now = {"device": 0}

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, now["device"] = now["device"], self.index

        def __exit__(self, *exc):
            now["device"] = self.before

    library = Library(now)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["device"])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(serving, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(serving, "_current_device", lambda: now["device"])
    monkeypatch.setattr(layers, "load_library", lambda path=None: library)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")                    # the address of a fake tensor is 0
        yield library, now


def t(dtype, *shape):
    return torch.empty(*shape, dtype=dtype, device="cuda:1")


bf16, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
CALLS = {
    "fp8_quantize_weight_device": lambda: ((t(f32, 2, 256, 128),), dict(transposed=True)),
    "fp8_gemm": lambda: ((t(u8, 5, 256), t(u8, 2, 5), t(u8, 130, 256), t(u8, 2, 2), t(bf16, 5, 130)), {}),
    "fp8_linear": lambda: ((t(f32, 5, 256), t(u8, 130, 256), t(u8, 2, 2), t(bf16, 5, 130)), dict(bias=t(f32, 130))),
    "fp8_linear_backward": lambda: ((t(bf16, 5, 144), t(bf16, 5, 256), t(u8, 256, 144), t(u8, 2, 2)),
                                    dict(dx=t(bf16, 5, 256), dw=t(f32, 144, 256), dbias=t(f32, 144), accumulate=True)),
    "residual_norm": lambda: ((t(bf16, 5, 33), t(f32, 5, 33), t(f32, 33)), dict(gate=t(f32, 5, 1))),
    "residual_norm_fp8": lambda: ((t(bf16, 5, 48), t(f32, 5, 48), t(f32, 48)), dict(gate=t(f32, 48))),
    "residual_norm_backward": lambda: ((t(f32, 5, 33), t(bf16, 5, 33), t(f32, 5, 33), t(bf16, 5, 33), t(f32, 2, 5), t(f32, 33)),
                                       dict(dy=t(bf16, 5, 33))),
    "moe_balance_loss": lambda: ((t(bf16, 5, 9), t(i32, 5, 2)), dict(seq_offsets=t(i32, 4))),
    "moe_router_backward": lambda: ((t(bf16, 5, 9), t(i32, 5, 2), t(bf16, 5, 9)), dict(dweights=t(f32, 5, 2))),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_tensors_gpu(name, current, world):
    library, now = world
    now["device"] = current
    args, more = CALLS[name]()
    getattr(gfg, name)(*args, **more)
    assert library.seen == [(name, 1, 0)] and now["device"] == current


@pytest.mark.parametrize("name", CALLS)
def test_calls_refuse_another_gpus_stream(name, world):
    library, _ = world

    class Other:
        cuda_stream, device = 0x1000, torch.device("cuda:0")

    args, more = CALLS[name]()
    with pytest.raises(ValueError, match="stream"):
        getattr(gfg, name)(*args, **more, stream=Other)
    assert not library.seen


@pytest.mark.parametrize("name,change", [
    ("fp8_gemm", {1: lambda: t(u8, 1, 5)}), ("fp8_gemm", {1: lambda: t(u8, 5, 2).t()}), ("fp8_gemm", {3: lambda: t(u8, 2, 1)}), ("fp8_gemm", {0: lambda: t(bf16, 5, 256)}),
    ("fp8_gemm", {4: lambda: t(f32, 5, 130)}), ("fp8_gemm", {1: lambda: torch.empty(2, 5, dtype=u8, device="cuda:0")}), ("fp8_linear", {0: lambda: t(f32, 256, 5).t()}),
    ("fp8_linear_backward", {1: lambda: t(f32, 5, 256)}), ("fp8_linear_backward", {2: lambda: t(u8, 144, 256)}), ("residual_norm", {1: lambda: t(torch.float16, 5, 33)}),
    ("residual_norm", {0: lambda: t(bf16, 5, 34)}), ("residual_norm_backward", {4: lambda: t(f32, 5, 2)}), ("residual_norm_backward", {1: lambda: t(torch.float16, 5, 33)}),
    ("moe_balance_loss", {1: lambda: t(torch.int64, 5, 2)}), ("moe_router_backward", {2: lambda: t(f32, 5, 9)}),
])
def test_calls_refuse_other_tensors(name, change, world):
    library, _ = world
    args, more = CALLS[name]()
    args = [change[i]() if i in change else a for i, a in enumerate(args)]
    with pytest.raises((TypeError, ValueError)):
        getattr(gfg, name)(*args, **more)
    assert not library.seen


# ------------------------------------------------------------------ the definitions
def directional(f, inputs, grads, seed):
    """f's change along a random direction, by central differences, and what the gradients say of it."""
    r = np.random.default_rng(seed)
    d = [r.standard_normal(np.shape(x)) for x in inputs]
    h = 1e-5
    diff = (f(*(x + h * v for x, v in zip(inputs, d))) - f(*(x - h * v for x, v in zip(inputs, d)))) / (2 * h)
    return diff, sum(float((g * v).sum()) for g, v in zip(grads, d))


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norm_gradients_against_differences(post, gate):
    r = np.random.default_rng(3)
    M, H, eps, alpha = 5, 17, 1e-3, 0.7
    y, res, w = r.standard_normal((M, H)), r.standard_normal((M, H)), r.standard_normal(H)
    wp = r.standard_normal(H) if post else None
    g = {"none": None, "channel": r.standard_normal(H), "token": r.standard_normal((M, 1))}[gate]
    dout, dz = r.standard_normal((M, H)), r.standard_normal((M, H))
    out, _, ry, ro = lo.residual_norm(y, res, w, wp, g, alpha, eps)
    grads = lo.residual_norm_backward(dout, dz, out, y, ry, ro, w, wp, g, alpha)
    names = [n for n, v in (("r", res), ("y", y), ("w", w), ("p", wp), ("g", g)) if v is not None]

    def loss(*v):
        a = dict(zip(names, v))
        o, z, _, _ = lo.residual_norm(a["y"], a["r"], a["w"], a.get("p"), a.get("g"), alpha, eps)
        return (o * dout).sum() + (z * dz).sum()

    inputs = [v for v in (res, y, w, wp, g) if v is not None]
    diff, said = directional(loss, inputs, [v for v in grads if v is not None], 4)
    assert abs(diff - said) <= 1e-7 * max(1.0, abs(diff))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("offsets", [None, [0, 4, 4, 11]])
def test_router_gradients_against_differences(score, renormalize, offsets):
    r = np.random.default_rng(5)
    T, E, k = 11, 7, 3
    logits = r.standard_normal((T, E))
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[2] = -1                                            # padding
    ids[5, 1] = E                                          # another rank's
    ids[6] = 4                                             # the same expert three times
    dw, dloss = r.standard_normal((T, k)), 1.7

    def loss(l):
        value = lo.balance(l, ids, score, 0.3, 0.05, offsets)[0]
        return dloss * value + (dw * lo.topk_weights(l, ids, score, renormalize, 2.5)).sum()

    factors = lo.balance(logits, ids, score, 0.3, 0.05, offsets)[2]
    d = lo.router_backward(logits, ids, dw, score, renormalize, 2.5, factors, dloss, offsets)
    diff, said = directional(loss, [logits], [d], 6)
    assert abs(diff - said) <= 1e-7 * max(1.0, abs(diff))


def test_balance_definition_example():
    """Two experts, every token on the first, even probabilities: f = (2, 0), P = (1/2, 1/2), loss alpha."""
    loss, counts, factors = lo.balance(np.zeros((4, 2)), np.zeros((4, 1), int), alpha=0.5, z=1.0)
    assert np.isclose(loss, 0.5 + np.log(2.0) ** 2) and counts.tolist() == [[4, 0]]
    assert np.allclose(factors, [[0.25, 0.0, 0.5]])


def test_linear_definition_example():
    """1 x 3 in E4M3: 1 and -3 are exact, 0.3 at scale 2^-7 (448 * 2^-7 = 3.5) is 38.4 -> 40 -> 0.3125."""
    y = lo.linear(np.array([[1.0, -3.0, 0.3]], np.float32), np.eye(3), [0.0, 0.0, 1.0])
    assert y.tolist() == [[1.0, -3.0, 1.3125]]
