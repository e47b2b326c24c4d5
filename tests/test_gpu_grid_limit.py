"""The grid limit on the integer products and the expert layer: what the launches ask for, read back from a captured
graph's kernel nodes, and that the results do not change."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_block_scaled_amd as gfg

pytestmark = pytest.mark.gpu


class Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class KernelNodeParams(ctypes.Structure):                  # hipKernelNodeParams
    _fields_ = [("blockDim", Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("gridDim", Dim3),
                ("kernelParams", ctypes.c_void_p), ("sharedMemBytes", ctypes.c_uint)]


def hip():
    """The HIP runtime that this process has loaded."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libamdhip64.so" in line}
    assert len(paths) == 1, paths
    return ctypes.CDLL(paths.pop())


def launches(call):
    """(workgroups, threads of a workgroup) of the kernels that call(stream) launches; nothing runs."""
    h, stream = hip(), torch.cuda.Stream()
    graph, n = ctypes.c_void_p(), ctypes.c_size_t()
    handle = ctypes.c_void_p(stream.cuda_stream)
    assert h.hipStreamBeginCapture(handle, 2) == 0         # relaxed
    try:
        call(stream)
    finally:
        assert h.hipStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert h.hipGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert h.hipGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        p = KernelNodeParams()
        assert h.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        out.append((p.gridDim.x * p.gridDim.y * p.gridDim.z, p.blockDim.x * p.blockDim.y * p.blockDim.z))
    assert h.hipGraphDestroy(graph) == 0
    return out


@pytest.fixture(params=[8, 24, 56])
def limit(request):
    yield request.param
    gfg.set_grid_limit(0)
    gfg.set_tile_shape(gfg.TILE_AUTO)


def codes(gen, *shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=gen)


def scales(gen, *shape):
    return (torch.rand(*shape, device="cuda", generator=gen) + 0.5) / 1000


def both(limit, call, out):
    """The result without a limit and, over the same garbage, with it; and what the limited call launches."""
    call(None)
    torch.cuda.synchronize()
    want = out.clone()
    out.fill_(7.0)
    gfg.set_grid_limit(limit)
    got = launches(call)
    torch.cuda.synchronize()
    call(None)
    torch.cuda.synchronize()
    return want, got


# one size for each kernel: 16 x 32 and 32 x 32 tiles, 64 x 64, 128 x 128, the large ones
@pytest.mark.parametrize("M,N,K", [(16, 3000, 272), (32, 2900, 400), (100, 1999, 272), (600, 1900, 144), (1900, 1500, 272), (2100, 2050, 272)])
@pytest.mark.parametrize("small", [True, False])
def test_dense(M, N, K, small, limit):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    a, b, sa, sb = codes(gen, M, K), codes(gen, N, K), scales(gen, M), scales(gen, N)
    d = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    gfg.set_tile_shape(gfg.TILE_128x256 if small else gfg.TILE_AUTO)
    want, got = both(limit, lambda s: gfg.int8_gemm(a, sa, b, sb, d, stream=s), d)
    assert len(got) == 1 and got[0][0] <= limit, got
    assert torch.equal(d, want)


@pytest.mark.parametrize("M", [1, 2, 3, 4])
def test_linear_of_a_few_tokens(M, limit):
    N, K = 2500, 1040
    gen = torch.Generator(device="cuda").manual_seed(M)
    b, sb, x = codes(gen, N, K), scales(gen, N), torch.randn(M, K, device="cuda", generator=gen)
    d = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gfg.int8_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    want, got = both(limit, lambda s: gfg.int8_linear(x, b, sb, d, workspace=ws, stream=s), d)
    assert max(g for g, _ in got) <= limit, got
    assert torch.equal(d, want)


@pytest.mark.parametrize("rows", [[100, 1, 128, 0, 300], [16, 9, 40, 128], [900, 5, 256]])
@pytest.mark.parametrize("masked", [False, True])
def test_grouped(rows, masked, limit):
    G, N, K = len(rows), 1100, 272
    gen = torch.Generator(device="cuda").manual_seed(sum(rows))
    b, sb = codes(gen, G, N, K), scales(gen, G, N)
    gfg.set_tile_shape(gfg.TILE_128x256)
    if masked:
        top = max(rows)
        a, sa, meta = codes(gen, G, top, K), scales(gen, G, top), torch.tensor(rows, dtype=torch.int32, device="cuda")
        d = torch.zeros(G, top, N, dtype=torch.float16, device="cuda")
        fn = gfg.grouped_int8_gemm_masked
    else:
        layout = np.concatenate([np.r_[np.full(m, g), np.full(-m % 128, -1)] for g, m in enumerate(rows)]).astype(np.int32)
        M = layout.size
        a, sa, meta = codes(gen, M, K), scales(gen, M), torch.from_numpy(layout).cuda()
        d = torch.zeros(M, N, dtype=torch.float16, device="cuda")
        fn = gfg.grouped_int8_gemm_contiguous
    d.fill_(7.0)                                           # rows of no expert keep it
    want, got = both(limit, lambda s: fn(a, sa, b, sb, meta, d, stream=s), d)
    assert len(got) == 1 and got[0][0] <= limit, got
    assert torch.equal(d, want)


# resident and streamed token rows, units of few and of many rows, the down projection in one launch and in two
@pytest.mark.parametrize("T,E,k,H,I", [(1, 16, 8, 1024, 512), (17, 8, 3, 2048, 256), (100, 8, 1, 4096, 1792), (150, 6, 2, 384, 1536)])
def test_layer(T, E, k, H, I, limit):
    """The sums of a hidden value may be added in another order, so results agree to roundings: the outputs' own (2^-8,
    one a side), and 2^-12 of a row's largest output for everything before it."""
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    w1, s1, w2, s2 = codes(gen, E, 2 * I, H), scales(gen, E, 2 * I), codes(gen, E, H, I), scales(gen, E, H)
    x = torch.randn(T, H, device="cuda", generator=gen).to(torch.bfloat16)
    ids = torch.rand(T, E, device="cuda", generator=gen).argsort(-1)[:, :k].int().contiguous()
    w = torch.rand(T, k, device="cuda", generator=gen)
    out = torch.zeros_like(x)
    ws = torch.empty(gfg.moe_layer_workspace_bytes(T, k, H, I), dtype=torch.uint8, device="cuda")
    want, got = both(limit, lambda s: gfg.moe_int8_layer(x, ids, w, w1, s1, w2, s2, out, workspace=ws, stream=s), out)
    products = [g for g, threads in got if threads == 512]
    assert len(products) == 2 and max(products) <= limit, got
    a, b = out.double(), want.double()
    assert bool(((a - b).abs() <= 2 * 2.0 ** -8 * 1.01 * b.abs() + 2.0 ** -12 * b.abs().amax(1, keepdim=True)).all())
