"""The ragged products on the GPU against plain references in 64 bits.

Group sizes cover the empty group, one row, sizes on both sides of the tiles'
edges (16, 32, 128, 256 rows) and rows of no group; widths cover whole and
partial 64-, 128- and 256-column tiles, both weight layouts and element types,
and padded row pitches.  The bounds are derived in ragged_ref.
"""
import numpy as np
import pytest
import torch

import ragged_ref as ref
from tiled_dense_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tiled_dense_gemm_gb300 import build
    build.build()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.synchronize()


def normal(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).to(DEV)


def offsets_of(sizes, head=0):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + head).to(DEV).contiguous()


def weights(G, K, N, layout, seed, dtype, scale):
    return normal((G, K, N) if layout == "kn" else (G, N, K), seed, dtype, scale)


# (rows of each group, rows before the first, rows after the last)
GROUPS = [
    ([1], 0, 0),
    ([0], 0, 3),
    ([3, 0, 1, 16, 17, 0], 0, 0),
    ([15, 33, 31, 64, 65, 0, 127], 2, 5),
    ([0, 0, 128, 129, 0], 0, 0),
    ([255, 257, 0, 300], 0, 1),
    ([512, 1, 0, 513], 7, 0),
    ([600], 0, 0),
    ([2] * 40, 0, 0),
]
SIZES = [(8, 8), (64, 64), (128, 256), (136, 520), (1000, 264), (392, 72), (2056, 136)]


@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "f16"), ("kn", "bf16"), ("nk", "bf16")])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "-".join(map(str, g[0][:7])))
def test_grouped(groups, layout, dtype):
    sizes, head, tail = groups
    T = head + sum(sizes) + tail
    off = offsets_of(sizes, head)
    for i, (K, N) in enumerate(SIZES):
        if sum(sizes) > 500 and K * N > 200000:
            continue
        x, w = normal((T, K), 10 + i, dtype), weights(len(sizes), K, N, layout, 20 + i, dtype, K ** -0.5)
        for relu in (True, False):
            y = binding.gemm_relu_grouped(x, w, off, apply_relu=relu, b_layout=layout)
            binding.check_device_error()
            ref.check(y, ref.grouped(x, w, off, relu, layout), f"{sizes} {K}x{N} {layout} {dtype} relu={relu}")


@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "f16"), ("kn", "bf16"), ("nk", "bf16")])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "-".join(map(str, g[0][:7])))
def test_grouped_dx(groups, layout, dtype):
    sizes, head, tail = groups
    T = head + sum(sizes) + tail
    off = offsets_of(sizes, head)
    for i, (N, K) in enumerate(SIZES):
        if sum(sizes) > 500 and K * N > 200000:
            continue
        dy, w = normal((T, N), 30 + i, dtype), weights(len(sizes), K, N, layout, 40 + i, dtype, N ** -0.5)
        act = torch.relu(normal((T, K), 50 + i, dtype))
        for gate in (None, act):
            dx = binding.gemm_relu_grouped_dx(dy, w, off, act=gate, b_layout=layout)
            binding.check_device_error()
            ref.check(dx, ref.grouped_dx(dy, w, off, gate, layout), f"{sizes} {K}x{N} {layout} {dtype} {gate is not None}")


@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "f16"), ("kn", "bf16"), ("nk", "bf16")])
@pytest.mark.parametrize("groups", GROUPS, ids=lambda g: "-".join(map(str, g[0][:7])))
def test_grouped_dw(groups, layout, dtype):
    sizes, head, tail = groups
    T = head + sum(sizes) + tail
    off = offsets_of(sizes, head)
    for i, (K, N) in enumerate(SIZES):
        x, dy = normal((T, K), 60 + i, dtype), normal((T, N), 70 + i, dtype)
        dw = binding.gemm_relu_grouped_dw(x, dy, off, b_layout=layout)
        binding.check_device_error()
        ref.check(dw, ref.grouped_dw(x, dy, off, layout), f"{sizes} {K}x{N} {layout} {dtype}")


IDS = [
    (1, 1, "one"), (1, 3, "none"), (5, 2, "mixed"), (16, 16, "each"), (40, 7, "mixed"), (64, 64, "each"),
    (100, 3, "runs"), (129, 4, "runs"), (300, 9, "mixed"), (300, 2, "none"), (520, 5, "runs"), (257, 100, "mixed"),
]


def make_ids(T, R, kind, seed):
    rs = np.random.RandomState(seed)
    if kind == "none":
        ids = np.full(T, -1)
    elif kind == "one":
        ids = np.zeros(T)
    elif kind == "each":
        ids = rs.permutation(R)[:T]
    elif kind == "mixed":
        ids = rs.randint(-1, R, T)
    else:
        ids = np.repeat(rs.randint(-1, R, (T + 36) // 37), 37)[:T]
    return torch.from_numpy(ids.astype(np.int32)).to(DEV)


@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "f16"), ("kn", "bf16"), ("nk", "bf16")])
@pytest.mark.parametrize("rank", [1, 8, 16, 20, 64, 72, 128])
def test_adapters(rank, layout, dtype):
    for i, (T, R, kind) in enumerate(IDS):
        K, N = SIZES[(i + rank) % len(SIZES)]
        x, a, b = normal((T, K), 80 + i, dtype), normal((R, rank, K), 90 + i, dtype, K ** -0.5), normal((R, rank, N), 95 + i, dtype, rank ** -0.5)
        w = normal((K, N) if layout == "kn" else (N, K), 85 + i, dtype, K ** -0.5)
        ids = make_ids(T, R, kind, i)
        scale = (torch.rand(R, generator=torch.Generator().manual_seed(i)) + 0.5).to(DEV)
        for relu, s in ((True, scale), (False, None)):
            y = binding.gemm_relu_adapters(x, w, a, b, ids, s, apply_relu=relu, b_layout=layout)
            binding.check_device_error()
            ref.check(y, ref.adapters(x, w, a, b, ids, s, relu, layout), f"T={T} R={R} {kind} {K}x{N} rank {rank} {layout} {dtype}")


@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "bf16")])
@pytest.mark.parametrize("T,R,rank,kind", [(1025, 3, 16, "runs"), (1500, 40, 12, "mixed"), (2500, 5, 96, "runs")])
def test_adapters_many_rows(T, R, rank, kind, layout, dtype):
    K, N = 264, 328
    x, a, b = normal((T, K), 1, dtype), normal((R, rank, K), 2, dtype, K ** -0.5), normal((R, rank, N), 3, dtype, rank ** -0.5)
    w = normal((K, N) if layout == "kn" else (N, K), 4, dtype, K ** -0.5)
    ids = make_ids(T, R, kind, 5)
    scale = (torch.rand(R, generator=torch.Generator().manual_seed(6)) + 0.5).to(DEV)
    y = binding.gemm_relu_adapters(x, w, a, b, ids, scale, apply_relu=True, b_layout=layout)
    binding.check_device_error()
    ref.check(y, ref.adapters(x, w, a, b, ids, scale, True, layout), f"T={T} R={R} rank {rank} {kind} {layout} {dtype}")
