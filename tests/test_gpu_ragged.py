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


NAN_GROUPS = [[1, 2, 3], [15, 17, 1], [100, 28, 129], [127, 1, 128, 130], [40, 300, 5]]


@pytest.mark.parametrize("sizes", NAN_GROUPS, ids=str)
@pytest.mark.parametrize("K,N", [(72, 136), (520, 648)])
def test_rows_of_other_groups_do_not_enter(sizes, K, N):
    """NaN in one group's rows, in rows of no group and in one group's weights
    stays in that group's results."""
    for dtype in ("f16", "bf16"):
        T = sum(sizes) + 9
        off = offsets_of(sizes, 4)
        o = off.cpu().tolist()
        x, dy = normal((T, K), 1, dtype), normal((T, N), 2, dtype)
        w = weights(len(sizes), K, N, "kn", 3, dtype, K ** -0.5)
        for sick in range(len(sizes)):
            xs, ds, ws = x.clone(), dy.clone(), w.clone()
            for t in (xs, ds):
                t[:o[0]] = float("nan")
                t[o[-1]:] = float("inf")
                t[o[sick]:o[sick + 1]] = float("nan")
            ws[sick] = float("nan")
            y = binding.gemm_relu_grouped(xs, ws, off, apply_relu=False)
            dx = binding.gemm_relu_grouped_dx(ds, ws, off)
            dw = binding.gemm_relu_grouped_dw(xs, ds, off)
            binding.check_device_error()
            ry, rx, rw = (ref.grouped(x, w, off, False, "kn"), ref.grouped_dx(dy, w, off, None, "kn"),
                          ref.grouped_dw(x, dy, off, "kn"))
            rows = np.ones(T, bool)
            rows[o[sick]:o[sick + 1]] = False
            assert torch.isnan(y[~torch.from_numpy(rows).to(DEV)]).all()
            assert torch.isnan(dw[sick]).all()
            keep = torch.from_numpy(rows).to(DEV)
            ref.check(y[keep], (ry[0][rows], ry[1][rows]), f"y {sizes} {sick}")
            ref.check(dx[keep], (rx[0][rows], rx[1][rows]), f"dx {sizes} {sick}")
            others = [g for g in range(len(sizes)) if g != sick]
            ref.check(dw[others], (rw[0][others], rw[1][others]), f"dw {sizes} {sick}")
            assert (y[:o[0]] == 0).all() and (y[o[-1]:] == 0).all()


def test_gate_values():
    """The gate opens for positive numbers and +inf only, and a closed gate
    gives +0 whatever the product is."""
    for dtype in ("f16", "bf16"):
        K, N, T = 64, 64, 40
        off = offsets_of([17, 23])
        dy, w = normal((T, N), 1, dtype), weights(2, K, N, "kn", 2, dtype, N ** -0.5)
        act = normal((T, K), 3, dtype)
        special = [0.0, -0.0, float("inf"), float("-inf"), float("nan"), -1.0, 2.0 ** -14, -(2.0 ** -14)]
        for i, v in enumerate(special):
            act[:, i] = v
        value, bound = ref.grouped_dx(dy, w, off, None, "kn")
        dx = binding.gemm_relu_grouped_dx(dy, w, off, act=act)
        binding.check_device_error()
        keep = (act.double() > 0).cpu().numpy()
        ref.check(dx, (np.where(keep, value, 0.0), np.where(keep, bound, 0.0)), dtype)
        assert not torch.signbit(dx[~torch.from_numpy(keep).to(DEV)]).any()
        dy[:] = float("nan")
        dx = binding.gemm_relu_grouped_dx(dy, w, off, act=act)
        assert torch.isnan(dx[torch.from_numpy(keep).to(DEV)]).all()
        assert (dx[~torch.from_numpy(keep).to(DEV)] == 0).all()


def test_binding_refuses_on_the_gpu():
    x, w, off = normal((6, 64), 1, "f16"), weights(2, 64, 72, "kn", 2, "f16", 0.1), offsets_of([2, 4])
    call = binding.gemm_relu_grouped
    with pytest.raises(TypeError):
        call(x, w, off.long())
    with pytest.raises(ValueError):
        call(x, w, off[:2])
    with pytest.raises(ValueError):
        call(x, w, off.cpu())
    with pytest.raises(ValueError):
        call(x, w.transpose(1, 2), off, b_layout="nk")  # not contiguous
    with pytest.raises(ValueError):
        call(x.t().contiguous().t(), w, off)            # rows not contiguous
    with pytest.raises(ValueError):
        call(x, w, off, y=normal((6, 64), 3, "f16"))
    with pytest.raises(TypeError):
        call(x, w, off, y=normal((6, 72), 3, "bf16"))
    with pytest.raises(binding.GemmReluError):          # a pitch that is not a multiple of 16 bytes
        call(normal((6, 68), 4, "f16")[:, :64], w, off)
    with pytest.raises(binding.GemmReluError):          # rows that begin off a 16-byte boundary
        call(normal((6, 80), 4, "f16")[:, 4:68], w, off)
    with pytest.raises(ValueError):
        binding.gemm_relu_grouped_dx(normal((6, 72), 5, "f16"), w, off, act=normal((6, 72), 6, "f16"))
    with pytest.raises(ValueError):
        binding.gemm_relu_grouped_dw(x, normal((6, 72), 5, "f16"), off, dw=normal((2, 72, 64), 6, "f16"))
    a, b = normal((3, 4, 64), 7, "f16"), normal((3, 4, 72), 8, "f16")
    ids = torch.zeros(6, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        binding.gemm_relu_adapters(x, w[0], a, b, ids, torch.ones(3, device=DEV, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.gemm_relu_adapters(x, w[0], a, b, ids, torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        binding.gemm_relu_adapters(x, w[0], a, b, ids[:5])
    with pytest.raises(ValueError):
        binding.gemm_relu_adapters(x, w[0], a, b[:, :2], ids)
    binding.check_device_error()


@pytest.mark.parametrize("bad", [[0, 9, 5, 20], [-3, 4, 8, 20], [0, 4, 8, 99], [5, 5, 2, 1]])
def test_bad_offsets_are_reported(bad):
    """Offsets that decrease or leave [0, T]: reported once, nothing outside
    the outputs is written, and the next call is right."""
    T, K, N = 20, 72, 136
    x, dy, w = normal((T, K), 1, "f16"), normal((T, N), 2, "f16"), weights(3, K, N, "kn", 3, "f16", 0.1)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    good = offsets_of([3, 0, 17])
    guard = torch.full((3, T, N), 7.0, dtype=torch.float16, device=DEV)
    for run in (lambda o: binding.gemm_relu_grouped(x, w, o, y=guard[1]),
                lambda o: binding.gemm_relu_grouped_dx(dy, w, o),
                lambda o: binding.gemm_relu_grouped_dw(x, dy, o)):
        run(off)
        with pytest.raises(binding.GemmReluError, match="GEMM_ERR_INDEX"):
            binding.check_device_error()
        run(good)
        binding.check_device_error()
    assert (guard[0] == 7).all() and (guard[2] == 7).all()
    ref.check(guard[1], ref.grouped(x, w, good, True, "kn"), "after")


@pytest.mark.parametrize("T", [5, 200, 1300])
def test_bad_ids_are_reported(T):
    R, rank, K, N = 3, 8, 64, 72
    x, a, b, w = normal((T, K), 1, "f16"), normal((R, rank, K), 2, "f16", 0.1), normal((R, rank, N), 3, "f16"), normal((K, N), 4, "f16", 0.1)
    ids = make_ids(T, R, "mixed", 1)
    sick = ids.clone()
    sick[1], sick[T - 1] = R, -2
    y = binding.gemm_relu_adapters(x, w, a, b, sick)
    with pytest.raises(binding.GemmReluError, match="GEMM_ERR_INDEX"):
        binding.check_device_error()
    none = sick.clone()
    none[1] = none[T - 1] = -1
    ref.check(y, ref.adapters(x, w, a, b, none, None, True, "kn"), "as without adapter")
    y = binding.gemm_relu_adapters(x, w, a, b, ids)
    binding.check_device_error()
    ref.check(y, ref.adapters(x, w, a, b, ids, None, True, "kn"), "after")


@pytest.mark.parametrize("T", [7, 130, 700, 1100])
def test_adapters_do_not_mix(T):
    """A NaN factor or an infinite scale of one adapter stays in its rows."""
    R, rank, K, N = 5, 20, 136, 200
    x, a, b, w = normal((T, K), 1, "bf16"), normal((R, rank, K), 2, "bf16", 0.1), normal((R, rank, N), 3, "bf16"), normal((K, N), 4, "bf16", 0.1)
    scale = torch.ones(R, device=DEV)
    ids = make_ids(T, R, "mixed", 2)
    rows = (ids != 1) & (ids != 3) & (ids != 4)
    value, bound = ref.adapters(x, w, a, b, ids, scale, False, "kn")
    a[1], b[3], scale[4] = float("nan"), float("nan"), float("inf")
    y = binding.gemm_relu_adapters(x, w, a, b, ids, scale, apply_relu=False)
    binding.check_device_error()
    keep = rows.cpu().numpy()
    ref.check(y[rows], (value[keep], bound[keep]), f"T={T}")
    assert torch.isnan(y[(ids == 1) | (ids == 3)]).all()


def test_row_pitches():
    """Rows inside wider matrices, for every row operand; what lies between
    them is neither read nor written."""
    T, K, N, sizes = 70, 72, 136, [30, 0, 33]
    off = offsets_of(sizes, 2)
    def padded(width, seed, left):
        wide = torch.full((T, width + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
        wide[:, left:left + width] = normal((T, width), seed, "bf16")
        return wide[:, left:left + width], wide
    x, _ = padded(K, 1, 8)
    dy, _ = padded(N, 2, 16)
    act, _ = padded(K, 3, 0)
    w = weights(3, K, N, "kn", 4, "bf16", 0.1)
    y, wide_y = padded(N, 5, 8)
    binding.gemm_relu_grouped(x, w, off, y=y)
    ref.check(y, ref.grouped(x, w, off, True, "kn"), "y")
    dx, wide_dx = padded(K, 6, 16)
    binding.gemm_relu_grouped_dx(dy, w, off, act=act, dx=dx)
    ref.check(dx, ref.grouped_dx(dy, w, off, act, "kn"), "dx")
    ref.check(binding.gemm_relu_grouped_dw(x, dy, off), ref.grouped_dw(x, dy, off, "kn"), "dw")
    a, b = normal((4, 12, K), 7, "bf16", 0.1), normal((4, 12, N), 8, "bf16")
    ids = make_ids(T, 4, "mixed", 9)
    y2, wide_y2 = padded(N, 10, 8)
    binding.gemm_relu_adapters(x, w[0], a, b, ids, y=y2)
    ref.check(y2, ref.adapters(x, w[0], a, b, ids, None, True, "kn"), "adapters")
    binding.check_device_error()
    for wide, left, width in ((wide_y, 8, N), (wide_dx, 16, K), (wide_y2, 8, N)):
        assert torch.isnan(wide[:, :left]).all() and torch.isnan(wide[:, left + width:]).all()


def test_sums_of_nothing_and_of_one():
    """No group, no reduction, no row: zeros; outputs of stale memory are overwritten."""
    K, N = 64, 72
    x, w = normal((5, K), 1, "f16"), weights(2, K, N, "kn", 2, "f16", 0.1)
    y = torch.full((5, N), 9.0, dtype=torch.float16, device=DEV)
    binding.gemm_relu_grouped(x, w[:0], offsets_of([]), y=y)
    assert (y == 0).all()
    y.fill_(9)
    binding.gemm_relu_grouped(x[:, :0], w[:, :0].contiguous(), offsets_of([2, 3]), y=y)
    assert (y == 0).all()
    dw = torch.full((2, K, N), 9.0, dtype=torch.float16, device=DEV)
    binding.gemm_relu_grouped_dw(x[:0], y[:0], offsets_of([0, 0]), dw=dw)
    assert (dw == 0).all()
    dw.fill_(9)
    binding.gemm_relu_grouped_dw(x, y, offsets_of([0, 0]), dw=dw)
    assert (dw == 0).all()
    assert binding.gemm_relu_grouped(x[:0], w, offsets_of([0, 0])).shape == (0, N)
    binding.check_device_error()


def test_every_group_count():
    """As many groups as a call takes, one row each but for a few."""
    G, K, N = 1024, 64, 64
    rs = np.random.RandomState(0)
    for sizes in (rs.randint(0, 3, G), rs.randint(0, 2, G) * 0, np.eye(1, G, 700, dtype=int)[0] * 150,
                  rs.randint(0, 300, G)):
        T = int(sizes.sum()) + 2
        off = offsets_of(sizes)
        x, dy, w = normal((T, K), 1, "f16"), normal((T, N), 2, "f16"), weights(G, K, N, "kn", 3, "f16", 0.1)
        ref.check(binding.gemm_relu_grouped(x, w, off), ref.grouped(x, w, off, True, "kn"), "y")
        ref.check(binding.gemm_relu_grouped_dw(x, dy, off), ref.grouped_dw(x, dy, off, "kn"), "dw")
        binding.check_device_error()


def _differences(f, t, h, picks, rs):
    """Central differences of the scalar f() in a few entries of t (float64)."""
    out = []
    flat = t.view(-1)
    for i in rs.choice(flat.numel(), picks, replace=False):
        v = flat[i].item()
        flat[i] = v + h
        up = f()
        flat[i] = v - h
        down = f()
        flat[i] = v
        out.append((int(i), (up - down) / (2 * h)))
    return out


def test_gradients_against_differences():
    """dx (through the ReLU below) and dw of L = sum(c * y), y = x w, x =
    ReLU(z), against central differences of L in 64 bits.  L is linear in w and
    piecewise linear in z, so a difference is exact up to rounding where z is
    further from 0 than the step."""
    rs = np.random.RandomState(3)
    T, K, N, sizes = 37, 64, 72, [5, 0, 20, 11]
    off = offsets_of(sizes)
    z = normal((T, K), 1, "f16")
    z[z.abs() < 2.0 ** -6] = 0.25
    x, w, c = torch.relu(z), weights(4, K, N, "kn", 2, "f16", 0.1), normal((T, N), 3, "f16")
    dx = binding.gemm_relu_grouped_dx(c, w, off, act=x).double().cpu().view(-1)
    dw = binding.gemm_relu_grouped_dw(x, c, off).double().cpu().view(-1)
    binding.check_device_error()
    z64, w64, c64 = z.double().cpu(), w.double().cpu(), c.double().cpu()
    bounds = ref.bounds_of(off, T)

    def loss():
        x64 = torch.relu(z64)
        return sum(float((c64[lo:hi] * (x64[lo:hi] @ w64[g])).sum()) for g, (lo, hi) in enumerate(bounds))

    _, bx = ref.grouped_dx(c, w, off, x, "kn")
    _, bw = ref.grouped_dw(x, c, off, "kn")
    h = 2.0 ** -8
    slack = 64 * T * N * K * 2.0 ** -53 / h  # rounding of the two sums, of terms of order one
    for i, d in _differences(loss, z64, h, 60, rs):
        assert abs(d - dx[i].item()) <= bx.reshape(-1)[i] + slack
    for i, d in _differences(loss, w64, h, 60, rs):
        assert abs(d - dw[i].item()) <= bw.reshape(-1)[i] + slack


def test_two_streams_and_a_graph():
    """Calls on two streams at once keep apart; a captured sequence replays on
    new inputs and offsets in the same buffers."""
    T, K, N, R, rank = 300, 264, 520, 6, 16
    w = weights(5, K, N, "kn", 1, "bf16", K ** -0.5)
    a, b = normal((R, rank, K), 2, "bf16", K ** -0.5), normal((R, rank, N), 3, "bf16", rank ** -0.5)

    def inputs(seed):
        rs = np.random.RandomState(seed)
        sizes = rs.multinomial(T - 3, np.ones(5) / 5)
        return normal((T, K), seed, "bf16"), normal((T, N), seed + 1, "bf16"), offsets_of(sizes, 1), make_ids(T, R, "mixed", seed)

    def run(x, dy, off, ids):
        return (binding.gemm_relu_grouped(x, w, off), binding.gemm_relu_grouped_dx(dy, w, off, act=x),
                binding.gemm_relu_grouped_dw(x, dy, off), binding.gemm_relu_adapters(x, w[0], a, b, ids),
                binding.gemm_relu_adapters(x[:40], w[0], a, b, ids[:40].contiguous()))

    def check(out, x, dy, off, ids, what):
        ref.check(out[0], ref.grouped(x, w, off, True, "kn"), what)
        ref.check(out[1], ref.grouped_dx(dy, w, off, x, "kn"), what)
        ref.check(out[2], ref.grouped_dw(x, dy, off, "kn"), what)
        ref.check(out[3], ref.adapters(x, w[0], a, b, ids, None, True, "kn"), what)
        ref.check(out[4], ref.adapters(x[:40], w[0], a, b, ids[:40], None, True, "kn"), what)

    sets = [inputs(10), inputs(20)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(run(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            check(o, *sets[i], f"stream {i}")
            assert all(torch.equal(p, q) for p, q in zip(o, outs[i][0]))
    held = [t.clone() for t in sets[0]]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(*held)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = run(*held)
    for new in (sets[1], sets[0], inputs(30)):
        for t, n in zip(held, new):
            t.copy_(n)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(out, *new, "replay")
    binding.check_device_error()


def test_results_do_not_change_from_run_to_run():
    for T, G in ((40, 6), (3000, 9)):
        K, N = 392, 520
        rs = np.random.RandomState(T)
        off = offsets_of(rs.multinomial(T, np.ones(G) / G))
        x, dy, w = normal((T, K), 1, "f16"), normal((T, N), 2, "f16"), weights(G, K, N, "nk", 3, "f16", K ** -0.5)
        a, b, ids = normal((7, 24, K), 4, "f16", K ** -0.5), normal((7, 24, N), 5, "f16"), make_ids(T, 7, "mixed", 6)
        runs = [(binding.gemm_relu_grouped(x, w, off, b_layout="nk"), binding.gemm_relu_grouped_dx(dy, w, off, b_layout="nk"),
                 binding.gemm_relu_grouped_dw(x, dy, off, b_layout="nk"),
                 binding.gemm_relu_adapters(x, w[0], a, b, ids, b_layout="nk")) for _ in range(5)]
        for r in runs[1:]:
            assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


def test_results_past_32_bit_offsets():
    """Outputs and weights of more than 2^32 bytes and 2^31 elements: the last
    rows of Y and the last expert, against those rows alone."""
    K, N, T = 64, 4096, (1 << 31) // 4096 + 300
    w = weights(3, K, N, "kn", 1, "f16", K ** -0.5)
    off = torch.tensor([0, 5, T - 200, T], dtype=torch.int32, device=DEV)
    x = torch.randn(T, K, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).half()
    y = binding.gemm_relu_grouped(x, w, off)
    binding.check_device_error()
    tail = x[T - 400:].contiguous()
    ref.check(y[T - 400:], ref.grouped(tail, w, torch.tensor([0, 0, 200, 400]), True, "kn"), "tail")
    ref.check(y[:8], ref.grouped(x[:8].contiguous(), w, torch.tensor([0, 5, 8, 8]), True, "kn"), "head")
    del y, x
    G, K, N = 600, 1024, 4096  # 2.5e9 elements of weights
    w = torch.zeros((G, K, N), dtype=torch.float16, device=DEV)
    w[-1] = normal((K, N), 3, "f16", K ** -0.5)
    x = normal((40, K), 4, "f16")
    off = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    off[-1] = 40
    y = binding.gemm_relu_grouped(x, w, off)
    ref.check(y, ref.grouped(x, w[-1:], torch.tensor([0, 40]), True, "kn"), "last expert")
    dw = binding.gemm_relu_grouped_dw(x, y, off, dw=w)
    ref.check(dw[-1:], ref.grouped_dw(x, y, torch.tensor([0, 40]), "kn"), "last gradient")
    assert not dw[:-1].any()
    binding.check_device_error()


def test_example_block():
    """The example's block, forward and backward, against plain 64-bit torch
    with autograd; the library's outputs that are rounded on the way (h, u, z,
    dz, du) set the tolerance: their unit roundoff, a few times over."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")
    spec = importlib.util.spec_from_file_location("expert_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for T in (6, 300):
        block = mod.ExpertBlock(136, 264, 8, 2, 4, 8, dtype=torch.float16, device=DEV, seed=T)
        x, dy = normal((T, 136), 1, "f16"), normal((T, 136), 2, "f16")
        ids = make_ids(T, 4, "mixed", 3)
        y, kept = block.forward(x, ids)
        dh, d_up, d_down = block.backward(dy, kept)
        binding.check_device_error()
        row, offsets, weight, rows, u, _ = kept
        h = torch.zeros((T, 136), dtype=torch.float64, device=DEV)
        h[row] = rows.double()
        h.requires_grad_()
        up, down = block.up.double().requires_grad_(), block.down.double().requires_grad_()
        out = torch.zeros((T, 136), dtype=torch.float64, device=DEV)
        for g, (lo, hi) in enumerate(ref.bounds_of(offsets, 2 * T)):
            z = torch.relu(h[row[lo:hi]] @ up[g]) @ down[g]
            out = out.index_add(0, row[lo:hi], z * weight[lo:hi, None].double())
        out.backward(dy.double())
        for got, want in ((y, out.detach()), (dh, h.grad), (d_up, up.grad), (d_down, down.grad)):
            off = (got.double() - want).norm() / want.norm()
            assert off < 8 * 2.0 ** -11, float(off)


@pytest.mark.parametrize("rank", [8, 40])
def test_adapters_do_not_mix_from_tile_to_tile(rank):
    """Many tiles per CTA, some with a factor that is not finite and some
    without: what one tile keeps out of its products the next does not."""
    T, K, N, R = 2304, 136, 8200, 6
    x, a, b, w = normal((T, K), 1, "bf16"), normal((R, rank, K), 2, "bf16", 0.1), normal((R, rank, N), 3, "bf16"), normal((K, N), 4, "bf16", 0.1)
    b[1, rank - 1, ::3] = float("inf")
    b[4, 0, 5000:] = float("nan")
    ids = (torch.arange(T, device=DEV) // 100 % R).int()
    ids[7::50] = 1
    ids[512:768] = 2
    ids[1500:1800] = -1
    y = binding.gemm_relu_adapters(x, w, a, b, ids, apply_relu=False)
    binding.check_device_error()
    rows = (ids != 1) & (ids != 4)
    value, bound = ref.adapters(x, w, a, torch.nan_to_num(b.float(), nan=0.0, posinf=0.0, neginf=0.0).to(b.dtype), ids, None, False, "kn")
    keep = rows.cpu().numpy()
    ref.check(y[rows], (value[keep], bound[keep]), f"rank {rank}")
    # and the broken rows have their own finite columns
    mine = (ids == 1).cpu().numpy()
    fine = np.ones(N, dtype=bool)
    fine[::3] = False
    ref.check(y[ids == 1][:, torch.from_numpy(fine).to(DEV)], (value[mine][:, fine], bound[mine][:, fine]), f"rank {rank}, finite columns")
    assert not torch.isfinite(y[ids == 1][:, ::3].float()).any()
    assert torch.isnan(y[ids == 4][:, 5000:].float()).all()


# Long groups with few tiles: clusters share the reduction, with shares that
# are empty (a short group beside long ones), and rows of no group that must not
# enter.
@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "bf16")])
@pytest.mark.parametrize("sizes,head,tail", [([2100], 0, 0), ([1500, 0, 1700], 5, 9), ([4111], 1, 0), ([3, 5000], 0, 130),
                                             ([130, 1, 3000, 700], 2, 0)], ids=str)
def test_grouped_dw_long(sizes, head, tail, layout, dtype):
    T = head + sum(sizes) + tail
    off = offsets_of(sizes, head)
    for i, (K, N) in enumerate([(8, 8), (136, 520), (392, 72), (256, 384), (1000, 264)]):
        x, dy = normal((T, K), 40 + i, dtype), normal((T, N), 50 + i, dtype)
        x[:head], dy[:head] = float("nan"), float("inf")
        x[T - tail:], dy[T - tail:] = float("inf"), float("nan")
        dw = binding.gemm_relu_grouped_dw(x, dy, off, b_layout=layout)
        binding.check_device_error()
        ref.check(dw, ref.grouped_dw(x, dy, off, layout), f"{sizes} {K}x{N} {layout} {dtype}")
        again = binding.gemm_relu_grouped_dw(x, dy, off, b_layout=layout)
        assert torch.equal(dw, again)


# Groups of many rows with many column tiles: CTA pairs (few tiles run as single
# CTAs), with the columns' last tile partial.
WIDE = [([255, 257, 0, 300], 0, 1), ([512, 1, 0, 513], 7, 0), ([600], 0, 0), ([33, 0, 410, 96, 31], 2, 2)]


@pytest.mark.parametrize("layout,dtype", [("kn", "f16"), ("nk", "f16"), ("kn", "bf16"), ("nk", "bf16")])
@pytest.mark.parametrize("groups", WIDE, ids=lambda g: "-".join(map(str, g[0])))
@pytest.mark.parametrize("K,N", [(136, 8200), (520, 5000), (1024, 4096)])
def test_grouped_wide(K, N, groups, layout, dtype):
    sizes, head, tail = groups
    T = head + sum(sizes) + tail
    off = offsets_of(sizes, head)
    x, w = normal((T, K), 31, dtype), weights(len(sizes), K, N, layout, 32, dtype, K ** -0.5)
    y = binding.gemm_relu_grouped(x, w, off, b_layout=layout)
    binding.check_device_error()
    ref.check(y, ref.grouped(x, w, off, True, layout), f"{sizes} {K}x{N} {layout} {dtype}")
    # the gradient with the same many columns: its reduction is the short side
    other = "nk" if layout == "kn" else "kn"
    w = weights(len(sizes), N, K, other, 33, dtype, K ** -0.5)
    act = normal((T, N), 34, dtype)
    dx = binding.gemm_relu_grouped_dx(x, w, off, act=act, b_layout=other)
    binding.check_device_error()
    ref.check(dx, ref.grouped_dx(x, w, off, act, other), f"dx {sizes} {K}x{N} {other} {dtype}")


# Bounded waits, by the library's own hook: the copy of one block of rows is
# left out, so a wait of the kernel runs out after a millisecond.  The sizes
# give plans of single CTAs without clusters.
HOOKED = {
    "grouped 0": (0, lambda x, w, g, off: binding.gemm_relu_grouped(x, w, off),
                  lambda x, w, g, off: ref.grouped(x, w, off, True, "kn")),
    "grouped 2": (2, lambda x, w, g, off: binding.gemm_relu_grouped(x, w, off),
                  lambda x, w, g, off: ref.grouped(x, w, off, True, "kn")),
    "dw 0": (0, lambda x, w, g, off: binding.gemm_relu_grouped_dw(x, g, off),
             lambda x, w, g, off: ref.grouped_dw(x, g, off, "kn")),
}


@pytest.mark.parametrize("what", list(HOOKED))
def test_timed_out_wait_is_reported_and_the_next_call_is_correct(what, monkeypatch):
    kb, call, want = HOOKED[what]
    sizes, K, N = [7, 0, 15, 8, 10], 512, 2048 if kb or "dw" not in what else 256
    off = offsets_of(sizes)
    x, w = normal((sum(sizes), K), 1, "f16"), weights(5, K, N, "kn", 2, "f16", K ** -0.5)
    g = normal((sum(sizes), N), 3, "f16")
    monkeypatch.setenv("GEMM_RELU_TEST_DROP_KB", str(kb))
    call(x, w, g, off)
    with pytest.raises(binding.GemmReluError) as e:
        binding.check_device_error()
    assert e.value.status == 6  # GEMM_ERR_TIMEOUT
    monkeypatch.delenv("GEMM_RELU_TEST_DROP_KB")
    binding.check_device_error()
    for _ in range(2):
        y = call(x, w, g, off)
        binding.check_device_error()
        ref.check(y, want(x, w, g, off), what)


def test_the_hook_is_refused_where_it_does_not_apply(monkeypatch):
    def refused(call):
        with pytest.raises(binding.GemmReluError) as e:
            call()
        assert e.value.status == 1  # GEMM_ERR_INVALID_ARG

    x, w = normal((40, 512), 1, "f16"), weights(5, 512, 2048, "kn", 2, "f16", 0.05)
    off = offsets_of([7, 0, 15, 8, 10])
    monkeypatch.setenv("GEMM_RELU_TEST_DROP_KB", "4")  # K = 512: k-blocks 0 .. 3
    refused(lambda: binding.gemm_relu_grouped(x, w, off))
    monkeypatch.setenv("GEMM_RELU_TEST_DROP_KB", "0")
    # clusters; pairs; adapters
    refused(lambda: binding.gemm_relu_grouped(x, w[:, :, :128].contiguous(), off))
    refused(lambda: binding.gemm_relu_grouped(normal((400, 512), 1, "f16"), w, offsets_of([100, 0, 100, 200, 0])))
    refused(lambda: binding.gemm_relu_adapters(
        x, w[0], normal((2, 8, 512), 1, "f16"), normal((2, 8, 2048), 1, "f16"),
        torch.zeros(40, dtype=torch.int32, device=DEV)))
    monkeypatch.delenv("GEMM_RELU_TEST_DROP_KB")
    binding.check_device_error()


def test_adapters_of_many_rows_on_two_streams_and_in_a_graph():
    """Calls whose low-rank products are tiles of their own, on two streams of
    unequal priority while a third one holds part of the GPU: each call ends
    whatever share of the GPU it gets, and its result is the one it has alone.
    Then the same calls captured, and replayed on other inputs."""
    K, N, R, rank = 264, 1032, 40, 40
    w, a, b = normal((K, N), 1, "bf16", K ** -0.5), normal((R, rank, K), 2, "bf16", K ** -0.5), normal((R, rank, N), 3, "bf16", rank ** -0.5)
    sets = [(normal((T, K), T, "bf16"), make_ids(T, R, "mixed", T)) for T in (1100, 2600)]
    alone = [binding.gemm_relu_adapters(x, w, a, b, ids) for x, ids in sets]
    binding.check_device_error()
    for (x, ids), y in zip(sets, alone):
        ref.check(y, ref.adapters(x, w, a, b, ids, None, True, "kn"), f"{len(ids)} rows")
    xd, wd = normal((2048, 2048), 4, "f16"), normal((2048, 1024), 5, "f16", 0.02)
    low, high = torch.cuda.Stream.priority_range()
    streams = [torch.cuda.Stream(priority=low), torch.cuda.Stream(priority=high)]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        with torch.cuda.stream(other):
            binding.gemm_relu(xd, wd)
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(binding.gemm_relu_adapters(sets[i][0], w, a, b, sets[i][1]))
    torch.cuda.synchronize()
    binding.check_device_error()
    for i in range(2):
        assert all(torch.equal(y, alone[i]) for y in outs[i])
    x, ids = (t.clone() for t in sets[0])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        binding.gemm_relu_adapters(x, w, a, b, ids)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y = binding.gemm_relu_adapters(x, w, a, b, ids)
            z = binding.gemm_relu_adapters(x, w, a, b, ids, apply_relu=False)
    x.copy_(sets[1][0][:1100])
    ids.copy_(sets[1][1][:1100])
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    binding.check_device_error()
    ref.check(y, ref.adapters(x, w, a, b, ids, None, True, "kn"), "replayed")
    ref.check(z, ref.adapters(x, w, a, b, ids, None, False, "kn"), "replayed, no ReLU")


@pytest.mark.parametrize("T,R,rank,kind", [(1100, 200, 512, "mixed"), (1400, 90, 136, "mixed"), (3000, 256, 8, "mixed"), (2300, 64, 24, "runs")])
def test_adapters_with_many_low_rank_tiles_per_block(T, R, rank, kind):
    """Tens of tiles of low-rank products on each pair of CTAs (200 adapters of
    rank 512 in each row tile), then several tiles of Y with as many extra
    k-blocks: every accumulator's turn is taken by the warps that release it.
    Five calls give the same bits."""
    K, N = 136, 72 if rank > 100 else 4104
    x, a, b = normal((T, K), 1, "bf16"), normal((R, rank, K), 2, "bf16", K ** -0.5), normal((R, rank, N), 3, "bf16", rank ** -0.5)
    w, ids = normal((K, N), 4, "bf16", K ** -0.5), make_ids(T, R, kind, 5)
    y = binding.gemm_relu_adapters(x, w, a, b, ids, apply_relu=False)
    binding.check_device_error()
    ref.check(y, ref.adapters(x, w, a, b, ids, None, False, "kn"), f"T={T} R={R} rank {rank}")
    for _ in range(4):
        assert torch.equal(y, binding.gemm_relu_adapters(x, w, a, b, ids, apply_relu=False))
    binding.check_device_error()


# (T > 128: pairs; rank 8 and an odd number of adapters in a row tile: a box of
# zeros pads the last extra k-block's products)
@pytest.mark.parametrize("T", [7, 128, 200, 1000, 1300])
@pytest.mark.parametrize("rank", [8, 5, 16, 24])
def test_ids_outside_the_range_count_as_none(T, rank):
    """Whatever value an id outside [-1, R) has, its row is one without
    adapter, also where an earlier call left NaN in the workspace."""
    for R in (1, 3):
        K, N = 64, 72
        for dtype in ("f16", "bf16"):
            x, a, b, w = normal((T, K), 1, dtype), normal((R, rank, K), 2, dtype, 0.1), normal((R, rank, N), 3, dtype), normal((K, N), 4, dtype, 0.1)
            ids = (torch.arange(T, device=DEV) % R).int()
            sick = ids.clone()
            bad = torch.tensor([-2, -3, -4, -5, R, R + 1, -(2 ** 31), 2 ** 31 - 1, -3, -3], dtype=torch.int32, device=DEV)
            at = torch.arange(T, device=DEV)[1::5]
            sick[at] = bad[torch.arange(len(at), device=DEV) % len(bad)]
            if T > 200:
                sick[40:90] = -3
            none = torch.where((sick >= 0) & (sick < R), sick, torch.full_like(sick, -1))
            binding.gemm_relu_adapters(x, w, torch.full_like(a, float("nan")), b, ids)  # NaN in every row's low-rank part
            y = binding.gemm_relu_adapters(x, w, a, b, sick, apply_relu=False)
            with pytest.raises(binding.GemmReluError, match="GEMM_ERR_INDEX"):
                binding.check_device_error()
            ref.check(y, ref.adapters(x, w, a, b, none, None, False, "kn"), f"T={T} R={R} rank {rank} {dtype}")


@pytest.mark.parametrize("what", ["grouped 0", "dw 0"])
def test_a_timeout_does_not_hide_bad_offsets(what, monkeypatch):
    """A launch whose wait runs out and that met offsets outside [0, T]: both
    are reported, the timeout first, each once."""
    kb, call, want = HOOKED[what]
    sizes, K, N = [7, 0, 15, 8, 10], 512, 2048 if "dw" not in what else 256
    off = offsets_of(sizes)
    x, w = normal((sum(sizes), K), 1, "f16"), weights(5, K, N, "kn", 2, "f16", K ** -0.5)
    g = normal((sum(sizes), N), 3, "f16")
    bad = off.clone()
    bad[-1] = 41  # one row more than there are
    monkeypatch.setenv("GEMM_RELU_TEST_DROP_KB", str(kb))
    call(x, w, g, bad)
    monkeypatch.delenv("GEMM_RELU_TEST_DROP_KB")
    for status in (6, 9):  # GEMM_ERR_TIMEOUT, GEMM_ERR_INDEX
        with pytest.raises(binding.GemmReluError) as e:
            binding.check_device_error()
        assert e.value.status == status
    binding.check_device_error()
    y = call(x, w, g, off)
    binding.check_device_error()
    ref.check(y, want(x, w, g, off), what)


@pytest.mark.parametrize("T", [5, 200, 1300])
@pytest.mark.parametrize("power", [-20, -14, -8, 12])
def test_small_and_large_low_rank_parts(T, power):
    """Scales of 2^power with second factors of 2^-power (2^12 at most: binary16): low is held to
    u^2 |low| or half the type's smallest step, and no better is promised; the
    bound takes that through |B|."""
    K, N, R, rank = 136, 264, 3, 12
    for dtype in ("f16", "bf16"):
        x, a, w = normal((T, K), 1, dtype), normal((R, rank, K), 2, dtype, K ** -0.5), normal((K, N), 4, dtype, 0.1)
        b = normal((R, rank, N), 3, dtype, 2.0 ** min(-power, 12))
        ids, scale = make_ids(T, R, "mixed", 5), torch.full((R,), 2.0 ** power, device=DEV)
        y = binding.gemm_relu_adapters(x, w, a, b, ids, scale, apply_relu=False)
        binding.check_device_error()
        ref.check(y, ref.adapters(x, w, a, b, ids, scale, False, "kn"), f"T={T} 2^{power} {dtype}")


def test_low_rank_parts_beyond_binary16():
    """From 65520 up low is infinite in binary16, for the rows of that adapter
    alone; bfloat16 holds it."""
    T, K, N, R, rank = 300, 64, 72, 2, 4
    for dtype in ("f16", "bf16"):
        x, a, w = normal((T, K), 1, dtype), normal((R, rank, K), 2, dtype, K ** -0.5), normal((K, N), 4, dtype, 0.1)
        x[:, 0], a[:, :, 0] = 1.0, 8.0  # low > 0 but for a few rows
        b = normal((R, rank, N), 3, dtype, 2.0 ** -14)
        ids = (torch.arange(T, device=DEV) % R).int()
        scale = torch.tensor([1.0, 2.0 ** 16], device=DEV)
        y = binding.gemm_relu_adapters(x, w, a, b, ids, scale, apply_relu=False)
        binding.check_device_error()
        value, bound = ref.adapters(x, w, a, b, ids, scale, False, "kn")
        if dtype == "bf16":
            ref.check(y, (value, bound), "bfloat16")
            continue
        ref.check(y[ids == 0], (value[::2], bound[::2]), "the other rows")
        low = (x.double() @ a[1].double().t() * 2.0 ** 16).abs()
        assert not torch.isfinite(y[(ids == 1) & (low > 65536).any(1)]).any()


@pytest.mark.parametrize("T", [262144, 262144 + 300])
def test_adapters_of_a_whole_block_of_rows_and_more(T):
    """As many row tiles as one launch lists, and rows that go on in a second
    block of them: the rows at both ends and on both sides of the seam."""
    K, N, R, rank = 64, 72, 5, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, K, generator=g, device=DEV).half()
    a, b, w = normal((R, rank, K), 2, "f16", K ** -0.5), normal((R, rank, N), 3, "f16", rank ** -0.5), normal((K, N), 4, "f16", K ** -0.5)
    ids = make_ids(T, R, "mixed", 5)
    y = binding.gemm_relu_adapters(x, w, a, b, ids)
    binding.check_device_error()
    for lo in (0, 131000, 262144 - 200, T - 400):
        rows = slice(lo, min(lo + 400, T))
        ref.check(y[rows], ref.adapters(x[rows], w, a, b, ids[rows], None, True, "kn"), f"rows from {lo}")
