"""On which GPU the torch-facing calls run.  CPU test: tensors of a second GPU without storage (fake tensors), a
current device that is a plain variable, and a library that records which device is current when it is entered."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp8_block_scaled_amd as gfg
from fp8_block_scaled_amd import serving

bf16, i8, u8, i32, f32 = torch.bfloat16, torch.int8, torch.uint8, torch.int32, torch.float32


class Library:
    """Every entry point returns 0 and notes (its name, the current device, the last argument: the stream)."""

    def __init__(self, now):
        self.now, self.seen = now, []

    def __getattr__(self, name):
        def entry(*args):
            self.seen.append((name, self.now["device"], args[-1]))
            return 0
        return entry


@pytest.fixture
def world(monkeypatch):
    now = {"device": 0}

    class Device:                                          # torch.cuda.device
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, now["device"] = now["device"], self.index

        def __exit__(self, *exc):
            now["device"] = self.before

    class Stream:                                          # the default stream: handle 0 on every device
        cuda_stream = 0

    lib = Library(now)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now["device"])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(serving, "_raw_stream", lambda index: 0)
    if hasattr(serving, "_current_device"):
        monkeypatch.setattr(serving, "_current_device", lambda: now["device"])
    monkeypatch.setattr(gfg, "load_library", lambda path=None: lib)
    monkeypatch.setattr(serving, "load_library", lambda path=None: lib)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")                    # the address of a fake tensor is 0
        yield lib, now


def t(dtype, *shape, device="cuda:1"):
    return torch.empty(*shape, dtype=dtype, device=device)


M, N, K, G, S, T, k, E, H, I = 256, 256, 256, 2, 2, 3, 2, 4, 128, 128
FP8 = lambda D: (t(u8, M, K), t(u8, S, M), t(u8, G, N, K), t(u8, G, N // 128, S), t(i32, M), D)
FP8M = lambda D: (t(u8, G, M, K), t(u8, G, S, M), t(u8, G, N, K), t(u8, G, N // 128, S), t(i32, G), D)
MX = lambda D, e=1: (t(u8, M, K // e), t(u8, K // 32, M), t(u8, G, N, K // e), t(u8, G, K // 32, N), t(i32, M), D)
MXM = lambda D, e=1: (t(u8, G, M, K // e), t(u8, G, K // 32, M), t(u8, G, N, K // e), t(u8, G, K // 32, N), t(i32, G), D)
LAYER = lambda w, s1, s2: (t(bf16, T, H), t(i32, T, k), t(f32, T, k), t(w, E, 2 * I, H), s1, t(w, E, H, I), s2, t(bf16, T, H))
CALLS = {
    "grouped_fp8_gemm_contiguous": lambda: FP8(t(bf16, M, N)),
    "grouped_fp8_gemm_masked": lambda: FP8M(t(bf16, G, M, N)),
    "grouped_fp8_gemm_silu_mul_contiguous": lambda: FP8(t(bf16, M, N // 2)),
    "grouped_fp8_gemm_silu_mul_masked": lambda: FP8M(t(bf16, G, M, N // 2)),
    "grouped_mxfp8_gemm_contiguous": lambda: MX(t(bf16, M, N)),
    "grouped_mxfp8_gemm_masked": lambda: MXM(t(bf16, G, M, N)),
    "grouped_mxfp4_gemm_contiguous": lambda: MX(t(bf16, M, N), 2),
    "grouped_mxfp4_gemm_masked": lambda: MXM(t(bf16, G, M, N), 2),
    "grouped_mxfp4_gemm_silu_mul_contiguous": lambda: MX(t(bf16, M, N // 2), 2),
    "grouped_mxfp4_gemm_silu_mul_masked": lambda: MXM(t(bf16, G, M, N // 2), 2),
    "fp8_quantize_act_1x128_device": lambda: (t(bf16, M, K),),
    "int8_quantize_token_device": lambda: (t(bf16, M, K),),
    "int8_gemm": lambda: (t(i8, M, K), t(f32, M), t(i8, N, K), t(f32, N), t(bf16, M, N)),
    "int8_linear": lambda: (t(bf16, M, K), t(i8, N, K), t(f32, N), t(bf16, M, N)),
    "grouped_int8_gemm_contiguous": lambda: (t(i8, M, K), t(f32, M), t(i8, G, N, K), t(f32, G, N), t(i32, M), t(bf16, M, N)),
    "grouped_int8_gemm_masked": lambda: (t(i8, G, M, K), t(f32, G, M), t(i8, G, N, K), t(f32, G, N), t(i32, G), t(bf16, G, M, N)),
    "moe_topk": lambda: (t(f32, T, E), t(i32, T, k), t(f32, T, k)),
    "moe_fp8_layer": lambda: LAYER(u8, t(u8, E, 2 * I // 128, H // 128), t(u8, E, H // 128, I // 128)),
    "moe_int8_layer": lambda: LAYER(i8, t(f32, E, 2 * I), t(f32, E, H)),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_their_tensors_gpu(name, current, world):
    lib, now = world
    now["device"] = current
    getattr(gfg, name)(*CALLS[name]())
    assert [(n, device) for n, device, _ in lib.seen] in ([(name, 1)], [(name.replace("_device", "") + "_device", 1)]), lib.seen
    assert lib.seen[0][2] == 0 and now["device"] == current    # the default stream; the caller's device is back


@pytest.mark.parametrize("name", CALLS)
def test_calls_refuse_another_gpus_stream(name, world):
    lib, _ = world

    class Other:
        cuda_stream, device = 0x1000, torch.device("cuda:0")

    with pytest.raises(ValueError, match="stream"):
        getattr(gfg, name)(*CALLS[name](), stream=Other)
    assert not lib.seen
