"""The ragged products' entry points without a GPU: argument checks of the C
ABI (before any CUDA call) and of the Python binding."""
import pytest
import torch

GOOD = 4096  # a 16-byte aligned fake address: never dereferenced on these paths


def grouped(L, X=GOOD, W=GOOD, Y=GOOD, off=GOOD, T=8, G=2, N=8, K=8, ldx=None, ldy=None, layout=0, dtype=0):
    return L.gemm_relu_grouped(X, W, Y, off, T, G, N, K, K if ldx is None else ldx, N if ldy is None else ldy, 1,
                               layout, dtype, None)


def grouped_dx(L, dY=GOOD, W=GOOD, dX=GOOD, off=GOOD, act=None, T=8, G=2, N=8, K=8, ld_dy=None, ld_dx=None,
               ld_act=0, layout=0, dtype=0):
    return L.gemm_relu_grouped_dx(dY, W, dX, off, act, T, G, N, K, N if ld_dy is None else ld_dy,
                                  K if ld_dx is None else ld_dx, ld_act, layout, dtype, None)


def grouped_dw(L, X=GOOD, dY=GOOD, dW=GOOD, off=GOOD, T=8, G=2, N=8, K=8, ldx=None, ld_dy=None, layout=0, dtype=0):
    return L.gemm_relu_grouped_dw(X, dY, dW, off, T, G, N, K, K if ldx is None else ldx,
                                  N if ld_dy is None else ld_dy, layout, dtype, None)


def adapters(L, X=GOOD, W=GOOD, A=GOOD, B=GOOD, ids=GOOD, scale=GOOD, Y=GOOD, T=8, N=8, K=8, R=2, rank=4, ldx=None,
             ldy=None, layout=0, dtype=0):
    return L.gemm_relu_adapters(X, W, A, B, ids, scale, Y, T, N, K, R, rank, K if ldx is None else ldx,
                                N if ldy is None else ldy, 1, layout, dtype, None)


@pytest.mark.parametrize("call", [grouped, grouped_dx, grouped_dw, adapters], ids=lambda f: f.__name__)
def test_sizes_types_and_layouts(gemm_lib, call):
    L = gemm_lib.lib()
    for bad in (dict(T=-1), dict(N=-8), dict(K=-8), dict(T=1 << 31), dict(N=1 << 31), dict(K=1 << 31),
                dict(layout=2), dict(layout=-1), dict(dtype=2), dict(W=None) if call is not grouped_dw else dict(dW=None)):
        assert call(L, **bad) == 1, bad
    for bad in (dict(N=12), dict(K=12)):
        assert call(L, **bad) == 2, bad
    if call is not adapters:
        assert call(L, G=-1) == 1 and call(L, G=1025) == 1
        assert call(L, off=None) == 1 and call(L, off=GOOD + 2) == 2
    else:
        assert call(L, R=0) == 1 and call(L, R=-1) == 1 and call(L, rank=0) == 1 and call(L, rank=513) == 1
        assert call(L, ids=None) == 1 and call(L, ids=GOOD + 2) == 2 and call(L, scale=GOOD + 1) == 2
        assert call(L, A=None) == 1 and call(L, B=None) == 1 and call(L, A=GOOD + 8) == 2 and call(L, B=GOOD + 2) == 2


@pytest.mark.parametrize("call,rows", [(grouped, {"X": "ldx", "Y": "ldy"}), (grouped_dx, {"dY": "ld_dy", "dX": "ld_dx"}),
                                       (grouped_dw, {"X": "ldx", "dY": "ld_dy"}), (adapters, {"X": "ldx", "Y": "ldy"})],
                         ids=lambda f: getattr(f, "__name__", ""))
def test_row_matrices(gemm_lib, call, rows):
    L = gemm_lib.lib()
    for name, ld in rows.items():
        assert call(L, **{name: None}) == 1
        assert call(L, **{name: GOOD + 2}) == 2
        assert call(L, **{ld: 0}) == 1    # shorter than the row
        assert call(L, **{ld: 12}) == 2   # not a multiple of 16 bytes
    if call is grouped_dx:
        assert call(L, act=GOOD + 4, ld_act=8) == 2
        assert call(L, act=GOOD, ld_act=0) == 1


MAX_ROWS = 2 ** 31 - 2 ** 26  # GEMM_RELU_MAX_ROWS


@pytest.mark.parametrize("call", [grouped, grouped_dx, grouped_dw], ids=lambda f: f.__name__)
def test_rows_whose_tiles_leave_32_bits(gemm_lib, call):
    """Row counts from which tile counts, widths or loop ends pass 2^31 on the
    device are refused before any launch, for any group count."""
    L = gemm_lib.lib()
    for T in (MAX_ROWS + 1, 2 ** 31 - 2 ** 23, 2 ** 31 - 128, 2 ** 31 - 1):
        for G in (1, 80, 1024):
            assert call(L, T=T, G=G) == 1, (T, G)
    if not torch.cuda.is_available():  # the checks pass, no device is found
        assert call(L, T=MAX_ROWS) == 3
    # what the kernels add to a row number, a group's length or its end: its
    # tiles (64 rows at least), a tile's width, a block of 128 rows, a grid
    assert MAX_ROWS + -(-MAX_ROWS // 64) + 256 < 2 ** 31


def test_adapters_take_rows_in_blocks(gemm_lib):
    """Adapters' rows go in blocks of their own, so their number is bounded by
    the dimensions' limit alone."""
    L = gemm_lib.lib()
    assert adapters(L, T=1 << 31) == 1
    if not torch.cuda.is_available():
        assert adapters(L, T=2 ** 31 - 1) == 3


def test_nothing_to_do_needs_no_pointer(gemm_lib):
    L = gemm_lib.lib()
    none = dict(X=None, W=None)
    assert grouped(L, T=0, Y=None, off=None, **none) == 0 and grouped(L, N=0, Y=None, off=None, **none) == 0
    assert grouped_dx(L, T=0, dY=None, W=None, dX=None, off=None) == 0
    assert grouped_dx(L, K=0, dY=None, W=None, dX=None, off=None) == 0
    for empty in (dict(G=0), dict(N=0), dict(K=0)):
        assert grouped_dw(L, X=None, dY=None, dW=None, off=None, **empty) == 0
    assert adapters(L, T=0, Y=None, A=None, B=None, ids=None, **none) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks behaviour without a GPU")
def test_no_device_is_reported(gemm_lib):
    L = gemm_lib.lib()
    for call in (grouped, grouped_dx, grouped_dw, adapters):
        assert call(L) == 3


def test_binding_refuses(gemm_lib):
    import tiled_dense_gemm_gb300 as fw
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(2, 8, 16, dtype=torch.float16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fw.gemm_relu_grouped(x, w, off)  # CPU tensors
    with pytest.raises(TypeError):
        fw.gemm_relu_grouped(x.float(), w, off)
    with pytest.raises(TypeError):
        fw.gemm_relu_grouped(x, w.to(torch.bfloat16), off)
    with pytest.raises(TypeError):
        fw.gemm_relu_grouped([1.0], w, off)
    with pytest.raises(ValueError):
        fw.gemm_relu_grouped(x, w, off, b_layout="tn")
    with pytest.raises(ValueError):
        fw.gemm_relu_grouped(x[0], w, off)
    with pytest.raises(ValueError):
        fw.gemm_relu_grouped_dx(x, w, off)
    with pytest.raises(ValueError):
        fw.gemm_relu_grouped_dw(x, x[:3], off)
    with pytest.raises(ValueError):
        fw.gemm_relu_adapters(x, w[0], w, w, off)
    with pytest.raises(TypeError):
        fw.gemm_relu_adapters(x, w[0], w.float(), w, off)
