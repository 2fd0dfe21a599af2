"""The losses' entry points without a GPU: argument checks of the C ABI (before
any CUDA call), the workspace's size, and the Python binding's checks."""
import pytest
import torch

GOOD = 4096  # a 256-byte aligned fake address: never dereferenced on these paths
SPACE = 1 << 40


def xent(L, X=GOOD, W=GOOD, y=GOOD, loss=GOOD, lse=GOOD, T=8, V=16, D=8, ldx=None, layout=1, dtype=0, ws=GOOD, size=SPACE):
    return L.gemm_relu_xent(X, W, y, loss, lse, T, V, D, D if ldx is None else ldx, layout, dtype, ws, size, None)


def xent_grad(L, X=GOOD, W=GOOD, y=GOOD, lse=GOOD, dloss=GOOD, step=1, dX=GOOD, dW=GOOD, T=8, V=16, D=8, ldx=None, ld_dx=None, layout=1,
              dtype=0, ws=GOOD, size=SPACE):
    return L.gemm_relu_xent_grad(X, W, y, lse, dloss, step, dX, dW, T, V, D, D if ldx is None else ldx, D if ld_dx is None else ld_dx, layout,
                                 dtype, ws, size, None)


def distill(L, X=GOOD, W=GOOD, ids=GOOD, logits=GOOD, tau=1.0, loss=GOOD, lse=GOOD, T=8, V=16, D=8, k=3, ldx=None, ld_ids=None, ld_logits=None,
            layout=1, dtype=0, kind=2, ws=GOOD, size=SPACE):
    return L.gemm_relu_distill(X, W, ids, logits, tau, loss, lse, T, V, D, k, D if ldx is None else ldx, k if ld_ids is None else ld_ids,
                               k if ld_logits is None else ld_logits, layout, dtype, kind, ws, size, None)


def distill_grad(L, X=GOOD, W=GOOD, ids=GOOD, logits=GOOD, tau=1.0, lse=GOOD, dloss=GOOD, step=1, dX=GOOD, dW=GOOD, T=8, V=16, D=8, k=3, ldx=None,
                 ld_ids=None, ld_logits=None, ld_dx=None, layout=1, dtype=0, kind=2, ws=GOOD, size=SPACE):
    return L.gemm_relu_distill_grad(X, W, ids, logits, tau, lse, dloss, step, dX, dW, T, V, D, k, D if ldx is None else ldx,
                                    k if ld_ids is None else ld_ids, k if ld_logits is None else ld_logits, D if ld_dx is None else ld_dx,
                                    layout, dtype, kind, ws, size, None)


CALLS = [xent, xent_grad, distill, distill_grad]
GRADS = [xent_grad, distill_grad]
TEACHER = [distill, distill_grad]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_sizes_types_and_layouts(gemm_lib, call):
    L = gemm_lib.lib()
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(V=0), dict(V=-8), dict(V=(1 << 24) + 1), dict(D=0), dict(D=-8), dict(D=(1 << 20) + 8), dict(D=1 << 31),
                dict(layout=2), dict(layout=-1), dict(dtype=2), dict(dtype=-1), dict(X=None), dict(W=None), dict(ws=None), dict(size=0), dict(size=100),
                dict(ldx=0)):
        assert call(L, **bad) == 1, bad
    for bad in (dict(D=12), dict(V=12, layout=0), dict(X=GOOD + 8), dict(W=GOOD + 2), dict(ldx=12), dict(ws=GOOD + 16)):
        assert call(L, **bad) == 2, bad
    name = "y" if call in (xent, xent_grad) else "ids"
    assert call(L, **{name: None}) == 1 and call(L, **{name: GOOD + 2}) == 2


@pytest.mark.parametrize("call", [xent, distill], ids=lambda f: f.__name__)
def test_losses(gemm_lib, call):
    L = gemm_lib.lib()
    for name in ("loss", "lse"):
        assert call(L, **{name: None}) == 1 and call(L, **{name: GOOD + 2}) == 2


@pytest.mark.parametrize("call", GRADS, ids=lambda f: f.__name__)
def test_gradients(gemm_lib, call):
    L = gemm_lib.lib()
    for name in ("lse", "dloss"):
        assert call(L, **{name: None}) == 1 and call(L, **{name: GOOD + 1}) == 2
    assert call(L, step=2) == 1 and call(L, step=-1) == 1
    assert call(L, dX=GOOD + 2) == 2 and call(L, dW=GOOD + 2) == 2 and call(L, ld_dx=4) == 1 and call(L, ld_dx=12) == 2
    assert call(L, dX=None, dW=None, ws=None, size=0) == 0  # nothing wanted
    assert call(L, dX=None, dW=None, T=0) == 0


@pytest.mark.parametrize("call", TEACHER, ids=lambda f: f.__name__)
def test_teacher(gemm_lib, call):
    L = gemm_lib.lib()
    for bad in (dict(k=0), dict(k=-1), dict(k=1025), dict(ld_ids=2), dict(ld_logits=2), dict(kind=3), dict(kind=-1), dict(logits=None), dict(tau=0.0),
                dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-45)):
        assert call(L, **bad) == 1, bad
    assert call(L, logits=GOOD + 2) == 2 and call(L, logits=GOOD + 1, kind=0) == 2


def test_nothing_to_do(gemm_lib):
    L = gemm_lib.lib()
    for call in (xent, distill):
        assert call(L, T=0, X=None, W=None, loss=None, lse=None, ws=None, size=0, **({"y": None} if call is xent else {"ids": None, "logits": None})) == 0


def test_workspace(gemm_lib):
    size = gemm_lib.lib().gemm_relu_loss_workspace
    for bad in ((-1, 8, 8, 0, 0), (8, 0, 8, 0, 0), (8, 8, 0, 0, 0), (8, 8, 8, -1, 0), (8, 8, 8, 1025, 0), ((1 << 24) + 1, 8, 8, 0, 0)):
        assert size(*bad) == -1, bad
    assert size(8, 8, 12, 0, 0) == -2
    for grad in (0, 1):
        assert size(0, 8, 8, 0, grad) == 0
        for T, V, D in ((1, 1, 8), (64, 131072, 4096), (129, 50021, 2056), (8192, 131072, 4096), (1 << 24, 1000, 64)):
            need = size(T, V, D, 0, grad)
            assert need > 0 and need % 256 == 0
            assert size(T, V, D, 5, grad) > need
    # the logits of 8192 rows would be 2 GiB: the gradients take a piece of them and dX in 32 bits
    assert size(8192, 131072, 4096, 0, 1) < (1 << 29) + 2 * 8192 * 4096 * 4
    assert size(8192, 131072, 4096, 0, 0) < 1 << 29
    # a forward call's rows come in blocks, shorter ones for many words
    assert size(1 << 20, 131072, 4096, 0, 0) == size(16384, 131072, 4096, 0, 0)
    assert size(1 << 20, 1 << 20, 4096, 0, 0) < 2 * size(2048, 1 << 20, 4096, 0, 0)


def test_binding_without_a_gpu(gemm_lib):
    x, w = torch.zeros(4, 16, dtype=torch.float16), torch.zeros(32, 16, dtype=torch.float16)
    y, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    ids, logits = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    calls = [lambda **k: gemm_lib.gemm_relu_xent(x, w, y, **k), lambda **k: gemm_lib.gemm_relu_xent_grad(x, w, y, f, f, **k),
             lambda **k: gemm_lib.gemm_relu_distill(x, w, ids, logits, **k), lambda **k: gemm_lib.gemm_relu_distill_grad(x, w, ids, logits, f, f, **k)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call(b_layout="nk")
        with pytest.raises(ValueError, match="b_layout"):
            call(b_layout="vd")
    with pytest.raises(TypeError):
        gemm_lib.gemm_relu_xent(x.float(), w, y, b_layout="nk")
    with pytest.raises(TypeError):
        gemm_lib.gemm_relu_xent(x, None, y, b_layout="nk")
    with pytest.raises(ValueError, match="2-D"):
        gemm_lib.gemm_relu_xent(x[0], w, y, b_layout="nk")
