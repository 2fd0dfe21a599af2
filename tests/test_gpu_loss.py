"""The losses over a vocabulary on the GPU against plain references in 64 bits.

Rows on both sides of the tiles' edges (8, 128, 256), words on both sides of a
chunk's (64) and a tile's, widths that are whole and partial k-blocks, both
weight layouts and element types, rows without a wanted word (none, some, all
but one, all).  The bounds are derived in loss_ref.
"""
import ctypes

import numpy as np
import pytest
import torch

import loss_ref as ref
from tiled_dense_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
BOTH = [("nk", "f16"), ("kn", "f16"), ("nk", "bf16"), ("kn", "bf16")]


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


def head(V, D, layout, seed, dtype, scale=None):
    return normal((V, D) if layout == "nk" else (D, V), seed, dtype, 2 * D ** -0.5 if scale is None else scale)


def dloss_of(T, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(T, generator=g) + 0.25).mul_(1.0 / max(T, 1)).to(DEV)


def xent(x, w, y, layout, what, dloss=None):
    """Both directions of one cross entropy, checked."""
    words = ref.words_of(targets=y)
    loss, lse = binding.gemm_relu_xent(x, w, y, b_layout=layout)
    binding.check_device_error()
    want, want_lse = ref.losses(x, w, words, layout)
    ref.check(loss, want, f"loss {what}")
    ref.check(lse, want_lse, f"lse {what}")
    dloss = dloss_of(x.shape[0], 9) if dloss is None else dloss
    dx, dw = binding.gemm_relu_xent_grad(x, w, y, lse, dloss, b_layout=layout)
    binding.check_device_error()
    want_dx, want_dw = ref.gradients(x, w, words, lse, dloss, layout)
    ref.check(dx, want_dx, f"dx {what}")
    ref.check(dw, want_dw, f"dw {what}")
    return loss, lse, dx, dw


def distill(x, w, ids, logits, tau, layout, what, dloss=None):
    words = ref.words_of(ids=ids, logits=logits, tau=tau)
    loss, lse = binding.gemm_relu_distill(x, w, ids, logits, tau, b_layout=layout)
    binding.check_device_error()
    want, want_lse = ref.losses(x, w, words, layout, tau, cross=False)
    ref.check(loss, want, f"loss {what}")
    ref.check(lse, want_lse, f"lse {what}")
    dloss = dloss_of(x.shape[0], 9) if dloss is None else dloss
    dx, dw = binding.gemm_relu_distill_grad(x, w, ids, logits, lse, dloss, tau, b_layout=layout)
    binding.check_device_error()
    want_dx, want_dw = ref.gradients(x, w, words, lse, dloss, layout, tau, cross=False)
    ref.check(dx, want_dx, f"dx {what}")
    ref.check(dw, want_dw, f"dw {what}")
    return loss, lse, dx, dw


ROWS = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513]
WORDS = {"nk": [1, 2, 63, 64, 65, 200, 255, 257, 1003], "kn": [8, 64, 72, 200, 256, 264, 1000]}
WIDTHS = [8, 64, 72, 136, 256, 520]


@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", ROWS)
def test_xent(T, layout, dtype):
    for i, V in enumerate(WORDS[layout]):
        D = WIDTHS[(i + T) % len(WIDTHS)]
        x, w = normal((T, D), T, dtype), head(V, D, layout, V, dtype)
        y = ref.make_targets(T, V, 5, (0.0, 0.4, 0.9)[(i + T) % 3]).to(DEV)
        xent(x, w, y, layout, f"T {T} V {V} D {D} {layout} {dtype}")


@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", [1, 5, 8, 31, 64, 100, 128, 129, 256, 300, 513])
def test_distill(T, layout, dtype):
    for i, V in enumerate(WORDS[layout]):
        D, k = WIDTHS[(i + T) % len(WIDTHS)], (1, 2, 5, 33, 64, 130)[(i + T) % 6]
        tau = (1.0, 2.0, 0.5, 1.7)[i % 4]
        x, w = normal((T, D), T, dtype), head(V, D, layout, V, dtype)
        ids, logits = ref.make_words(T, V, k, 6, (0.0, 0.3, 0.9)[(i + T) % 3])
        distill(x, w, ids.to(DEV), logits.to(DEV), tau, layout, f"T {T} V {V} D {D} k {k} tau {tau} {layout} {dtype}")


@pytest.mark.parametrize("T", [3, 140, 400])
def test_all_rows_but_one_and_all(T):
    """No row in use: zeros; one row in use, wherever it is: its own numbers alone."""
    V, D = 300, 136
    x, w = normal((T, D), 1, "bf16"), head(V, D, "nk", 2, "bf16")
    for only in (None, 0, T // 2, T - 1):
        y = torch.full((T,), -1, dtype=torch.int32)
        if only is not None:
            y[only] = 17
        out = xent(x, w, y.to(DEV), "nk", f"only {only}")
        rest = torch.ones(T, dtype=torch.bool)
        if only is not None:
            rest[only] = False
        for o in out[:3]:
            assert not o[rest.to(DEV)].any()
        if only is None:
            assert not out[3].any()
        ids = torch.full((T, 3), -1, dtype=torch.int32)
        if only is not None:
            ids[only] = torch.tensor([299, -1, 0])
        out = distill(x, w, ids.to(DEV), torch.ones(T, 3, device=DEV), 1.5, "nk", f"only {only}")
        if only is None:
            assert not any(o.any() for o in out)


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=torch.float16, device=DEV), head(100, 64, "nk", 1, "f16")
    y, f = torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, device=DEV)
    loss, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    assert loss.shape == lse.shape == (0,)
    dw = torch.full_like(w, float("nan"))
    dx, dw = binding.gemm_relu_xent_grad(x, w, y, f, f, dw=dw, b_layout="nk")
    assert dx.shape == (0, 64) and not dw.any()
    ids, logits = torch.empty(0, 4, dtype=torch.int32, device=DEV), torch.empty(0, 4, device=DEV)
    loss, lse = binding.gemm_relu_distill(x, w, ids, logits, b_layout="nk")
    dx, dw = binding.gemm_relu_distill_grad(x, w, ids, logits, f, f, dw=torch.full_like(w, float("nan")), b_layout="nk")
    assert loss.shape == (0,) and not dw.any()
    binding.check_device_error()


@pytest.mark.parametrize("T", [40, 300, 700])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_rows_not_in_use_do_not_enter(T, layout):
    """Whatever the rows without a target hold, in X, lse and dloss: bit for bit the same results."""
    V, D = 1000, 136
    x, w = normal((T, D), 1, "f16"), head(V, D, layout, 2, "f16")
    y = ref.make_targets(T, V, 3, 0.5).to(DEV)
    y[-1] = -1
    out = (y < 0)
    loss, lse, dx, dw = xent(x, w, y, layout, "clean")
    dloss = dloss_of(T, 9)
    for bad in (float("nan"), float("inf"), 60000.0):
        x2, lse2, d2 = x.clone(), lse.clone(), dloss.clone()
        x2[out], lse2[out], d2[out] = bad, bad, bad
        loss2, lse3 = binding.gemm_relu_xent(x2, w, y, b_layout=layout)
        dx2, dw2 = binding.gemm_relu_xent_grad(x2, w, y, lse2, d2, b_layout=layout)
        assert torch.equal(loss, loss2) and torch.equal(lse, lse3) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    ids, logits = ref.make_words(T, V, 6, 4, 0.5)
    ids, logits = ids.to(DEV), logits.to(DEV)
    one = distill(x, w, ids, logits, 2.0, layout, "clean")
    l2 = logits.clone()
    l2[ids < 0] = float("nan")
    x2 = x.clone()
    x2[(ids < 0).all(dim=1)] = float("nan")
    two = binding.gemm_relu_distill(x2, w, ids, l2, 2.0, b_layout=layout)
    two += binding.gemm_relu_distill_grad(x2, w, ids, l2, two[1], dloss, 2.0, b_layout=layout)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    binding.check_device_error()


@pytest.mark.parametrize("k", [1, 31, 32, 33, 127, 500, 1024])
def test_many_words(k):
    T, V, D = 37, 1500, 72
    x, w = normal((T, D), 1, "bf16"), head(V, D, "nk", 2, "bf16")
    ids, logits = ref.make_words(T, V, k, 3, 0.1)
    distill(x, w, ids.to(DEV), logits.to(DEV), 1.0, "nk", f"k {k}")
    ids[:] = torch.arange(k, dtype=torch.int32) % 7  # a few words, many times each, close together
    distill(x, w, ids.to(DEV), logits.to(DEV), 2.0, "nk", f"k {k}, the same words")


@pytest.mark.parametrize("T", [30, 260])
def test_words_in_one_half_of_every_tile(T):
    """Short reductions and words in every other chunk of 64 columns: one half of the epilogue's warps has all
    of them to deal with and falls behind the other by several tiles."""
    V, D, k = 20000, 8, 1024
    x, w = normal((T, D), 1, "bf16"), head(V, D, "nk", 2, "bf16")
    rs = np.random.RandomState(3)
    for first in (0, 64):
        ids = (rs.randint(0, V // 128, (T, k)) * 128 + first + rs.randint(0, 64, (T, k))).astype(np.int32)
        ids[:, : k // 2] = first + rs.randint(0, 64, (T, k // 2))  # half of them in the first tile
        ids = torch.from_numpy(np.minimum(ids, V - 1))
        logits = torch.from_numpy(rs.standard_normal((T, k)).astype(np.float32))
        distill(x, w, ids.to(DEV), logits.to(DEV), 1.5, "nk", f"T {T} from {first}")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T", [5, 100, 130, 300])
def test_tiles_of_every_width(T, layout):
    """Vocabularies whose tiles are as wide as fills the waves: ends inside a chunk of 64 words, and a last tile
    of any width; words at the tiles' edges."""
    D, k = 16, 12
    for V in (8008, 9744, 12345, 17000, 19001, 22000, 30011, 40000):
        V = V // 8 * 8 if layout == "kn" else V
        x, w = normal((T, D), 1, "f16"), head(V, D, layout, 2, "f16")
        y = ref.make_targets(T, V, 3, 0.1)
        y[0], y[-1] = V - 1, 0
        xent(x, w, y.to(DEV), layout, f"T {T} V {V}")
        ids, logits = ref.make_words(T, V, k, 4, 0.1)
        ids[1::2] = torch.arange(k, dtype=torch.int32) * 16 + (torch.arange(T, dtype=torch.int32)[1::2, None] * 61) % (V - 16 * k)
        distill(x, w, ids.to(DEV), logits.to(DEV), 2.0, layout, f"T {T} V {V}")


def test_teacher_logits():
    """Logits of -infinity have no weight; of the type's lowest value, alone or with others, they do as any;
    16-bit types, pitches."""
    T, V, D, k = 70, 500, 64, 9
    x, w = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16")
    ids, logits = ref.make_words(T, V, k, 3, 0.1)
    logits[::2, 1] = -float("inf")
    logits[5] = -float("inf")          # a row whose words all have weight 0: none
    logits[6] = torch.finfo(torch.float32).min
    logits[7, ::2] = torch.finfo(torch.float32).min
    logits[8] = 3e38
    for tau in (0.5, 3.0):
        out = distill(x, w, ids.to(DEV), logits.to(DEV), tau, "nk", f"tau {tau}")
        assert out[0][5] == 0 and out[1][5] == 0 and not out[2][5].any()
    for t in (torch.float16, torch.bfloat16):
        l = logits.clamp(-60000, 60000).to(t).to(DEV)
        wide_ids, wide = torch.full((T, k + 3), 12345678, dtype=torch.int32, device=DEV), torch.full((T, k + 5), float("nan"), dtype=t, device=DEV)
        wide_ids[:, :k], wide[:, :k] = ids.to(DEV), l
        a = distill(x, w, ids.to(DEV), l, 2.0, "nk", str(t))
        b = distill(x, w, wide_ids[:, :k], wide[:, :k], 2.0, "nk", f"{t}, pitch")
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_pitches_and_given_outputs():
    T, V, D = 150, 333, 72
    w, y = head(V, D, "nk", 2, "f16"), ref.make_targets(T, V, 3, 0.2).to(DEV)
    x = normal((T, D), 1, "f16")
    wide = torch.full((T, 2 * D), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, :D] = x
    loss, lse, dx, dw = xent(x, w, y, "nk", "dense")
    d = dloss_of(T, 9)
    l2, s2 = torch.full((T,), float("nan"), device=DEV), torch.full((T,), float("nan"), device=DEV)
    out = binding.gemm_relu_xent(wide[:, :D], w, y, loss=l2, lse=s2, b_layout="nk")
    assert out[0] is l2 and out[1] is s2 and torch.equal(l2, loss) and torch.equal(s2, lse)
    # outputs inside larger buffers, which stay as they were
    frame = torch.full((T + 2, 2 * D), 7.0, dtype=torch.float16, device=DEV)
    frame_w = torch.full((V + 2, D), 7.0, dtype=torch.float16, device=DEV)
    binding.gemm_relu_xent_grad(wide[:, :D], w, y, lse, d, dx=frame[1:-1, :D], dw=frame_w[1:-1], b_layout="nk")
    assert torch.equal(frame[1:-1, :D], dx) and torch.equal(frame_w[1:-1], dw)
    frame[1:-1, :D], frame_w[1:-1] = 7.0, 7.0
    assert (frame == 7).all() and (frame_w == 7).all()
    # one of the two gradients alone
    a, none = binding.gemm_relu_xent_grad(x, w, y, lse, d, want_dw=False, b_layout="nk")
    none2, b = binding.gemm_relu_xent_grad(x, w, y, lse, d, want_dx=False, b_layout="nk")
    assert none is None and none2 is None and torch.equal(a, dx) and torch.equal(b, dw)
    assert binding.gemm_relu_xent_grad(x, w, y, lse, d, want_dx=False, want_dw=False, b_layout="nk") == (None, None)
    binding.check_device_error()


@pytest.mark.parametrize("T", [1, 20, 32, 33, 100, 300])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_one_gradient_alone(T, layout):
    """dX or dW without the other: the same bits."""
    V, D, k = 2000, 200, 4
    x, w = normal((T, D), T, "f16"), head(V, D, layout, 2, "f16")
    y, (ids, logits), d = ref.make_targets(T, V, 3, 0.2).to(DEV), ref.make_words(T, V, k, 4, 0.2), dloss_of(T, 5)
    ids, logits = ids.to(DEV), logits.to(DEV)
    _, lse = binding.gemm_relu_xent(x, w, y, b_layout=layout)
    _, lse2 = binding.gemm_relu_distill(x, w, ids, logits, 2.0, b_layout=layout)
    for call in (lambda **a: binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout=layout, **a),
                 lambda **a: binding.gemm_relu_distill_grad(x, w, ids, logits, lse2, d, 2.0, b_layout=layout, **a)):
        dx, dw = call()
        one, none = call(want_dw=False)
        none2, two = call(want_dx=False)
        assert none is none2 is None and torch.equal(one, dx) and torch.equal(two, dw)
    binding.check_device_error()


def test_gradient_of_broadcast_losses():
    """One value for all rows (a mean's gradient): one element, or an expanded view, as that value in each row."""
    T, V, D = 200, 300, 64
    x, w, y = normal((T, D), 1, "bf16"), head(V, D, "nk", 2, "bf16"), ref.make_targets(T, V, 3, 0.2).to(DEV)
    _, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    one = torch.tensor([0.003], device=DEV)
    want = binding.gemm_relu_xent_grad(x, w, y, lse, one.repeat(T), b_layout="nk")
    for d in (one, one[0], one.expand(T)):
        got = binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout="nk")
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    xent(x, w, y, "nk", "one", dloss=one)
    # one row
    d = torch.tensor([0.5], device=DEV)
    xent(x[:1], w, y[:1].clamp(min=0), "nk", "one row", dloss=d)
    binding.check_device_error()


@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", [1, 20, 100, 300])
def test_words_that_are_all_but_certain(T, layout, dtype):
    """exp(z - lse) - 1 is far below what a truncated sum of z is off by."""
    V, D, k = 1000, 2048, 4
    w = head(V, D, "nk", 60 + T, dtype)
    y = ref.make_targets(T, V, 61 + T)
    rows = w[y.cuda().long()].float()
    x = (24 * rows / rows.pow(2).sum(dim=1, keepdim=True)).to(w.dtype)
    w = w if layout == "nk" else w.t().contiguous()
    W = w.double() if layout == "kn" else w.double().t()
    dloss = dloss_of(T, 62)
    for tau, words, call in (
            (1.0, ref.words_of(targets=y), lambda s: binding.gemm_relu_xent_grad(x, w, y.cuda(), s, dloss, b_layout=layout)),
            (0.75, None, None)):
        if words is None:
            ids, logits = ref.make_words(T, V, k, 63, few=0.0)
            ids[:, 0] = ids[:, 2] = y  # (q near 1, in two places)
            logits[:, 0], logits[:, 2], logits[:, 1], logits[:, 3] = 9.0, 9.5, -1.0, -2.0
            words = ref.words_of(ids=ids, logits=logits, tau=tau)
            i, l = ids.cuda(), logits.cuda()
            call = lambda s: binding.gemm_relu_distill_grad(x, w, i, l, s, dloss, tau, b_layout=layout)  # noqa: E731
        lse = torch.logsumexp(x.double() @ W / tau, dim=1).float()
        dx, dw = call(lse)
        binding.check_device_error()
        rx, rw = ref.gradients(x, w, words, lse, dloss, layout, tau, cross=tau == 1.0)
        ref.check(dx, rx, f"dx, tau {tau}")
        ref.check(dw, rw, f"dw, tau {tau}")


@pytest.mark.parametrize("size", [1e-20, 1e-8, 1.0, 1e4])
def test_sizes_of_the_losses_gradient(size):
    """Binary16 holds g times a power of two: small and large gradients lose nothing but what dx and dw round."""
    T, V, D = 150, 400, 72
    x, w, y = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16"), ref.make_targets(T, V, 3, 0.2).to(DEV)
    for dtype in ("f16", "bf16"):
        xent(x.to(DT[dtype]), w.to(DT[dtype]), y, "nk", f"{size} {dtype}", dloss=dloss_of(T, 4) * size)
    zero = torch.zeros(T, device=DEV)
    out = xent(x, w, y, "nk", "zero", dloss=zero)
    assert not out[2].any() and not out[3].any()


def test_logits_that_are_not_finite():
    T, V, D = 140, 200, 64
    x, w = normal((T, D), 1, "bf16"), head(V, D, "nk", 2, "bf16")
    y = ref.make_targets(T, V, 3).to(DEV)
    clean = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    for rows in (T, 20):
        x2 = x[:rows].clone()
        x2[3, 5] = float("nan")     # NaN logits
        x2[7, :] = 0
        x2[7, 0] = 3e38             # infinite ones of both signs, as W's signs fall
        w2 = w.clone()
        w2[:, 0] *= 8
        loss, lse = binding.gemm_relu_xent(x2, w2, y[:rows].contiguous(), b_layout="nk")
        assert torch.isnan(lse[3]) and torch.isnan(loss[3])
        assert lse[7] == float("inf")
        keep = torch.ones(rows, dtype=torch.bool, device=DEV)
        keep[3] = keep[7] = False
        words = ref.words_of(targets=y[:rows])
        x3 = torch.where(keep[:, None], x2, torch.zeros_like(x2))
        (value, bound), _ = ref.losses(x3, w2, words, "nk")
        k = keep.cpu().numpy()
        ref.check(loss[keep], (value[k], bound[k]), "finite rows")
    # every logit minus infinity but one
    x2 = torch.zeros((1, D), dtype=torch.bfloat16, device=DEV)
    x2[0, 0] = -3e38
    w2 = torch.zeros_like(w)
    w2[:, 0] = 8.0
    w2[11, 0] = 0.0
    loss, lse = binding.gemm_relu_xent(x2, w2, torch.tensor([11], dtype=torch.int32, device=DEV), b_layout="nk")
    assert lse[0] == 0 and loss[0] == 0
    again = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    assert all(torch.equal(a, b) for a, b in zip(clean, again))
    binding.check_device_error()


@pytest.mark.parametrize("T", [20, 200])
def test_words_outside_the_vocabulary_are_reported(T):
    V, D = 100, 64
    x, w = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16")
    y = ref.make_targets(T, V, 3, 0.2)
    none = y.clone()
    none[4], none[9] = -1, -1
    y[4], y[9] = V, 2 ** 31 - 1
    want = xent(x, w, none.to(DEV), "nk", "without")
    got = binding.gemm_relu_xent(x, w, y.to(DEV), b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="INDEX"):
        binding.check_device_error()
    got += binding.gemm_relu_xent_grad(x, w, y.to(DEV), want[1], dloss_of(T, 9), b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="INDEX"):
        binding.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ids, logits = ref.make_words(T, V, 5, 6, 0.1)
    none = ids.clone()
    none[3, 2], none[8, 0] = -1, -1
    ids[3, 2], ids[8, 0] = V, 2 ** 31 - 1
    want = distill(x, w, none.to(DEV), logits.to(DEV), 2.0, "nk", "without")
    got = binding.gemm_relu_distill(x, w, ids.to(DEV), logits.to(DEV), 2.0, b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="INDEX"):
        binding.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    binding.check_device_error()


def _big(T, V, D, dtype, layout, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, D), generator=g, device=DEV).to(DT[dtype])
    w = (torch.randn((V, D) if layout == "nk" else (D, V), generator=g, device=DEV) * 2 * D ** -0.5).to(DT[dtype])
    return x, w


@pytest.mark.parametrize("layout,V", [("nk", 140003), ("kn", 140008)])
def test_several_pieces(layout, V):
    """More logits than one piece of the vocabulary holds, the last piece shorter and odd."""
    T, D = 2100, 72
    x, w = _big(T, V, D, "bf16", layout, 1)
    y = ref.make_targets(T, V, 3, 0.03).to(DEV)
    y[0], y[1] = V - 1, 0
    loss, lse = binding.gemm_relu_xent(x, w, y, b_layout=layout)
    d = dloss_of(T, 9)
    dx, dw = binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout=layout)
    binding.check_device_error()
    W = w.double() if layout == "nk" else w.double().T
    z = x.double() @ W.T
    live = (y >= 0)
    zy = z.gather(1, y.clamp(min=0).long()[:, None])[:, 0]
    want = torch.where(live, torch.logsumexp(z, 1), 0.0)
    assert (lse.double() - want).abs().max() < 1e-4
    assert (loss.double() - torch.where(live, want - zy, 0.0)).abs().max() < 1e-4
    g = z.sub_(lse.double()[:, None]).exp_()
    g[torch.arange(T, device=DEV), y.clamp(min=0).long()] -= 1
    g *= torch.where(live, d, torch.zeros_like(d)).double()[:, None]
    # g and the results are rounded to 8 bits: 2^-8 of the terms' sizes each
    for got, want, size in ((dx, g @ W, g.abs() @ W.abs()), (dw if layout == "nk" else dw.T, g.T @ x.double(), g.abs().T @ x.double().abs())):
        assert ((got.double() - want).abs() <= 2.0 ** -7 * size + 2.0 ** -8 * want.abs() + 1e-12).all()


@pytest.mark.parametrize("T", [31, 128])
def test_several_pieces_of_few_rows(T):
    """More words than G has room for at up to 128 rows, certain ones among them in every piece."""
    V, D = 4200008 if T < 128 else 2200008, 16
    w, x = head(V, D, "nk", 70, "bf16"), normal((T, D), 71, "bf16")
    y = ref.make_targets(T, V, 72).cuda()
    y[: T // 2] = torch.linspace(0, V - 1, T // 2, device=DEV).int()
    x[: T // 2] = (40 * w[y[: T // 2].long()].float() / w[y[: T // 2].long()].float().pow(2).sum(dim=1, keepdim=True)).to(x.dtype)
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, dim=1).float()
    dloss = dloss_of(T, 73)
    dx, dw = binding.gemm_relu_xent_grad(x, w, y, lse, dloss, b_layout="nk")
    binding.check_device_error()
    rows, a = torch.arange(T, device=DEV), dloss.double()[:, None]
    ez = D * ref.E32 * (x.double().abs() @ w.double().abs().t())
    p = torch.exp(z - lse.double()[:, None])
    e = p * (ez + 2 * ref.E32 * (z.abs() + lse.double().abs()[:, None]) + 2 * ref.E32)
    e[rows, y.long()] = torch.where(p[rows, y.long()] > 0.501, ez[rows, y.long()] / D + 2 * ref.E32, e[rows, y.long()])
    size = p.clone()
    size[rows, y.long()] += 1
    p[rows, y.long()] -= 1
    u = 2.0 ** -8
    g, e = a * p, a * (e + 4 * ref.E32 * size)
    e += u ** (2 if T <= 32 else 1) * (g.abs() + e) + 2.0 ** -134
    del z, ez, p, size
    X, W, n = x.double(), w.double(), g.abs() + e
    # (dX's sums: 16 products and one truncation at a time)
    for out, value, bound in ((dw, g.t() @ X, e.t() @ X.abs() + T * ref.E32 * (n.t() @ X.abs())),
                              (dx, g @ W, e @ W.abs() + V / 16 * ref.E32 * (n @ W.abs()))):
        off = (out.double() - value).abs() - (bound + u * (value.abs() + bound) + 2.0 ** -134)
        assert off.max().item() <= 0.0


def test_more_rows_than_a_block():
    T, V, D = 16384 + 300, 300, 64
    x, w = _big(T, V, D, "f16", "nk", 1)
    y = ref.make_targets(T, V, 3, 0.3).to(DEV)
    loss, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    tail = 16384 - 100
    want, want_lse = ref.losses(x[tail:], w, ref.words_of(targets=y[tail:]), "nk")
    ref.check(loss[tail:], want, "loss")
    ref.check(lse[tail:], want_lse, "lse")
    ids, logits = ref.make_words(T, V, 6, 4, 0.2)
    ids, logits = ids.to(DEV), logits.to(DEV)
    loss, lse = binding.gemm_relu_distill(x, w, ids, logits, 2.0, b_layout="nk")
    want, want_lse = ref.losses(x[tail:], w, ref.words_of(ids=ids[tail:], logits=logits[tail:], tau=2.0), "nk", 2.0, False)
    ref.check(loss[tail:], want, "distill loss")
    ref.check(lse[tail:], want_lse, "distill lse")
    binding.check_device_error()


def test_many_words_and_blocks_of_rows():
    """A vocabulary so large that a forward call's rows go in blocks of 2048, the last one shorter."""
    T, V, D = 2048 + 2048 + 77, 1 << 20, 16
    x, w = _big(T, V, D, "bf16", "nk", 1)
    y = ref.make_targets(T, V, 3, 0.2).to(DEV)
    loss, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, 3, 4, 0.2))
    soft, lse_tau = binding.gemm_relu_distill(x, w, ids, logits, 2.0, b_layout="nk")
    binding.check_device_error()
    at = torch.tensor([0, 1, 1500, 2047, 2048, 2100, 4095, 4096, T - 1], device=DEV)
    z = x[at].double() @ w.double().T
    live = y[at] >= 0
    want = torch.where(live, torch.logsumexp(z, 1), 0.0)
    assert (lse[at].double() - want).abs().max() < 1e-4
    zy = z.gather(1, y[at].clamp(min=0).long()[:, None])[:, 0]
    assert (loss[at].double() - torch.where(live, want - zy, 0.0)).abs().max() < 1e-4
    live = (ids[at] >= 0).any(1)
    assert (lse_tau[at].double() - torch.where(live, torch.logsumexp(z / 2, 1), 0.0)).abs().max() < 1e-4
    has = ids[at] >= 0
    q = torch.softmax(torch.where(has, logits[at].double() / 2, -1e30), 1) * has
    p = (torch.log_softmax(z / 2, 1)).gather(1, ids[at].clamp(min=0).long())
    want = 4 * (torch.xlogy(q, q) - q * p).sum(1)
    assert (soft[at].double() - torch.where(live, want, 0.0)).abs().max() < 1e-3


def test_weights_past_32_bit_offsets():
    """2.5e9 weights: the words at the end count as those at the start."""
    T, V, D = 3, 600001, 4096
    w = torch.zeros((V, D), dtype=torch.float16, device=DEV)
    w[-70:] = normal((70, D), 1, "f16", 2 * D ** -0.5)
    x = normal((T, D), 2, "f16")
    y = torch.tensor([V - 1, V - 65, 5], dtype=torch.int32, device=DEV)
    loss, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
    z = x.double() @ w[-70:].double().T
    zeros = torch.full((T, 1), np.log(V - 70), dtype=torch.float64, device=DEV)
    want = torch.logsumexp(torch.cat([z, zeros], 1), 1)
    zy = torch.stack([z[0, 69], z[1, 5], torch.zeros((), dtype=torch.float64, device=DEV)])
    assert (lse.double() - want).abs().max() < 1e-4 and (loss.double() - (want - zy)).abs().max() < 1e-4
    dx, dw = binding.gemm_relu_xent_grad(x, w, y, lse, torch.ones(T, device=DEV), b_layout="nk")
    g = torch.exp(z - lse.double()[:, None])
    g[0, 69] -= 1
    g[1, 5] -= 1
    size = g.abs().T @ x.double().abs()
    # (g of a word is about 1e-6: below 2^-17 of the largest, still 11 bits in binary16; dw's smallest step is 2^-24)
    assert ((dw[-70:].double() - g.T @ x.double()).abs() <= 2.0 ** -9 * size + 2.0 ** -24).all()
    big = g.abs() @ w[-70:].double().abs()
    assert ((dx.double() - g @ w[-70:].double()).abs() <= 2.0 ** -9 * big + 2.0 ** -24).all()
    p = torch.exp(-lse.double())  # a zero logit's share
    want = (p[:, None] * x.double()).sum(0)
    assert ((dw[1000].double() - want).abs() <= 2.0 ** -9 * (p[:, None] * x.double().abs()).sum(0) + 2.0 ** -24).all()
    binding.check_device_error()


def test_two_streams_and_graphs():
    """Calls on two streams at once, and two graphs of one capture stream replayed at once on two streams,
    keep apart; replays follow new inputs, row counts among them."""
    V, D, k = 1003, 136, 5
    w = head(V, D, "nk", 1, "bf16")

    def inputs(seed, T=300):
        ids, logits = ref.make_words(T, V, k, seed, 0.2)
        return [normal((T, D), seed, "bf16"), ref.make_targets(T, V, seed, (0.0, 0.3, 0.8)[seed % 3]).to(DEV), ids.to(DEV),
                logits.to(DEV), dloss_of(T, seed)]

    def run(x, y, ids, logits, d):
        a = binding.gemm_relu_xent(x, w, y, b_layout="nk")
        b = binding.gemm_relu_distill(x, w, ids, logits, 2.0, b_layout="nk")
        return (*a, *binding.gemm_relu_xent_grad(x, w, y, a[1], d, b_layout="nk"), *b,
                *binding.gemm_relu_distill_grad(x, w, ids, logits, b[1], d, 2.0, b_layout="nk"))

    sets = [inputs(s) for s in (10, 20, 30, 31)]
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*sets[i]))
    # ... and by the stream argument
    loss, lse = binding.gemm_relu_xent(sets[0][0], w, sets[0][1], b_layout="nk", stream=streams[0])
    raw = binding.gemm_relu_xent(sets[0][0], w, sets[0][1], b_layout="nk", stream=streams[1].cuda_stream)
    default = binding.gemm_relu_xent(sets[0][0], w, sets[0][1], b_layout="nk", stream=0)
    torch.cuda.synchronize()
    assert torch.equal(default[0], want[0][0])
    assert torch.equal(loss, want[0][0]) and torch.equal(lse, want[0][1]) and torch.equal(raw[0], loss)
    for i in range(2):
        for o in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(o, want[i]))
    held = [[t.clone() for t in sets[i]] for i in range(2)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            outs.append(run(*held[i]))
        graphs.append(g)
    for a, b in ((0, 1), (2, 3), (1, 0)):
        for i, s in enumerate((a, b)):
            for t, n in zip(held[i], sets[s]):
                t.copy_(n)
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i, s in enumerate((a, b)):
            assert all(torch.equal(p, q) for p, q in zip(outs[i], want[s]))
    binding.check_device_error()


@pytest.mark.parametrize("T,k", [(1, 3), (30, 40), (100, 7), (200, 40)])
def test_replays_follow_new_inputs(T, k):
    """One call behind another in the same memory, nothing waited for in between: each reads its own inputs."""
    V, D = 2003, 136
    w = head(V, D, "nk", 1, "bf16")

    def inputs(seed):
        ids, logits = ref.make_words(T, V, k, seed, 0.1)
        return [normal((T, D), seed, "bf16"), ref.make_targets(T, V, seed, 0.1).to(DEV), ids.to(DEV), logits.to(DEV), dloss_of(T, seed)]

    def run(x, y, ids, logits, d):
        a = binding.gemm_relu_xent(x, w, y, b_layout="nk")
        b = binding.gemm_relu_distill(x, w, ids, logits, 1.5, b_layout="nk")
        return (*a, *binding.gemm_relu_xent_grad(x, w, y, a[1], d, b_layout="nk"), *b,
                *binding.gemm_relu_distill_grad(x, w, ids, logits, b[1], d, 1.5, b_layout="nk"))

    sets = [inputs(s) for s in range(40, 48)]
    want = []
    for s in sets:
        want.append(run(*s))
        torch.cuda.synchronize()
    held = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run(*held)
    got = []
    for _ in range(3):
        for s in sets:
            for t, n in zip(held, s):
                t.copy_(n)
            g.replay()
            got.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    binding.check_device_error()
    for i, o in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(o, want[i % len(sets)])), i


def test_two_threads():
    """Two host threads, each on its own stream, with calls of several launches between each other's."""
    import threading
    V, D = 1003, 136
    w = head(V, D, "nk", 1, "f16")
    sets = []
    for i, T in enumerate((100, 300)):
        sets.append((normal((T, D), i, "f16"), ref.make_targets(T, V, i, 0.3).to(DEV), dloss_of(T, i)))

    def run(x, y, d):
        loss, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
        return (loss, lse, *binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout="nk"))

    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    got, wrong = [[], []], []

    def work(i):
        try:
            with torch.cuda.device(DEV), torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i].append(run(*sets[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for i in range(2):
        assert len(got[i]) == 20 and all(torch.equal(p, q) for o in got[i] for p, q in zip(o, want[i]))
    binding.check_device_error()


def test_results_do_not_change_from_run_to_run():
    for T, V, D in ((3, 5000, 264), (700, 3000, 520)):
        x, w, y = normal((T, D), 1, "bf16"), head(V, D, "nk", 2, "bf16"), ref.make_targets(T, V, 3, 0.3).to(DEV)
        d = dloss_of(T, 4)
        runs = []
        for _ in range(5):
            loss, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
            runs.append((loss, lse, *binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout="nk")))
        for r in runs[1:]:
            assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


@pytest.mark.parametrize("T", [5, 100, 400])
def test_workspace(T):
    """What the workspace holds before a call does not matter, and nothing behind its size is touched."""
    V, D, k = 1003, 136, 7
    L = binding.lib()
    x, w, y = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16"), ref.make_targets(T, V, 3, 0.3).to(DEV)
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, k, 4, 0.2))
    d = dloss_of(T, 9)
    loss, lse, dx, dw = xent(x, w, y, "nk", "clean")
    other = distill(x, w, ids, logits, 2.0, "nk", "clean")
    s = torch.cuda.current_stream().cuda_stream
    for fill in (0xFF, 0x7B):
        for teacher in (False, True):
            for grad in (0, 1):
                need = L.gemm_relu_loss_workspace(T, V, D, k if teacher else 0, grad)
                space = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
                o = [torch.full_like(t, float("nan")) for t in ((dx, dw) if grad else (loss, lse))]
                p = [t.data_ptr() for t in o]
                if teacher:
                    tau = ctypes.c_float(2.0)
                    if grad:
                        rc = L.gemm_relu_distill_grad(x.data_ptr(), w.data_ptr(), ids.data_ptr(), logits.data_ptr(), tau, other[1].data_ptr(),
                                                      d.data_ptr(), 1, *p, T, V, D, k, D, k, k, D, 1, 0, 2, space.data_ptr(), need, s)
                    else:
                        rc = L.gemm_relu_distill(x.data_ptr(), w.data_ptr(), ids.data_ptr(), logits.data_ptr(), tau, *p, T, V, D, k, D, k, k,
                                                 1, 0, 2, space.data_ptr(), need, s)
                elif grad:
                    rc = L.gemm_relu_xent_grad(x.data_ptr(), w.data_ptr(), y.data_ptr(), lse.data_ptr(), d.data_ptr(), 1, *p, T, V, D, D, D,
                                               1, 0, space.data_ptr(), need, s)
                else:
                    rc = L.gemm_relu_xent(x.data_ptr(), w.data_ptr(), y.data_ptr(), *p, T, V, D, D, 1, 0, space.data_ptr(), need, s)
                assert rc == 0
                binding.check_device_error()
                want = (other if teacher else (loss, lse, dx, dw))[2 * grad:2 * grad + 2]
                assert all(torch.equal(a, b) for a, b in zip(o, want))
                assert (space[need:] == fill).all()


def test_gradients_against_differences():
    """dx and dw of sum(c * loss) against central differences of it in 64 bits, for both losses."""
    T, V, D, k, tau = 23, 150, 40, 4, 1.5
    x, w = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16")
    y = ref.make_targets(T, V, 3, 0.2).to(DEV)
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, k, 4, 0.2))
    c = dloss_of(T, 5) * T
    x64, w64, c64 = x.double().cpu(), w.double().cpu(), c.double().cpu().numpy()
    for cross in (True, False):
        words = ref.words_of(targets=y) if cross else ref.words_of(ids=ids, logits=logits, tau=tau)
        t = 1.0 if cross else tau
        if cross:
            _, lse = binding.gemm_relu_xent(x, w, y, b_layout="nk")
            dx, dw = binding.gemm_relu_xent_grad(x, w, y, lse, c, b_layout="nk")
        else:
            _, lse = binding.gemm_relu_distill(x, w, ids, logits, tau, b_layout="nk")
            dx, dw = binding.gemm_relu_distill_grad(x, w, ids, logits, lse, c, tau, b_layout="nk")
        binding.check_device_error()
        (vx, bx), (vw, bw) = ref.gradients(x, w, words, lse, c, "nk", t, cross)
        value = lambda: float((ref.losses(x64, w64, words, "nk", t, cross)[0][0] * c64).sum())  # noqa: B023,E731
        rs, h = np.random.RandomState(6), 2.0 ** -10
        for flat, got, bound in ((x64.view(-1), dx, bx), (w64.view(-1), dw, bw)):
            got = got.double().cpu().view(-1)
            for i in rs.choice(flat.numel(), 40, replace=False):
                v = float(flat[i])
                flat[i] = v + h
                up = value()
                flat[i] = v - h
                down = value()
                flat[i] = v
                # third derivatives of the losses are at most c (max |w| or |x|)^3, times h^2 / 6; rounding of the two sums
                slack = h * h * float(np.abs(c64).max()) * 5 ** 3 + 1e-10
                assert abs((up - down) / (2 * h) - got[i].item()) <= bound.reshape(-1)[i] + slack


def test_a_step_of_both_losses():
    """As a training step uses them: rows of a block, both losses over the same weights, the gradients added up
    and sent on through the grouped products' gradient."""
    T, V, D, H, k, tau = 260, 700, 136, 264, 6, 2.0
    x, wb, w = normal((T, D), 1, "bf16"), normal((2, D, H), 2, "bf16", D ** -0.5), head(V, H, "nk", 3, "bf16")
    off = torch.tensor([0, 100, T], dtype=torch.int32, device=DEV)
    y = ref.make_targets(T, V, 4, 0.3).to(DEV)
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, k, 5, 0.2))
    h = binding.gemm_relu_grouped(x, wb, off)
    hard, lse = binding.gemm_relu_xent(h, w, y, b_layout="nk")
    soft, lse_tau = binding.gemm_relu_distill(h, w, ids, logits, tau, b_layout="nk")
    one = torch.full((1,), 1.0 / T, device=DEV)
    dh1, dw1 = binding.gemm_relu_xent_grad(h, w, y, lse, one * 0.3, b_layout="nk")
    dh2, dw2 = binding.gemm_relu_distill_grad(h, w, ids, logits, lse_tau, one * 0.7, tau, b_layout="nk")
    dz = binding.gemm_relu_grouped_dx(dh1 + dh2, torch.eye(H, dtype=torch.bfloat16, device=DEV).expand(2, H, H).contiguous(), off, act=h)
    binding.check_device_error()
    # the same with autograd in 64 bits
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    z = h64 @ w64.T
    live = y >= 0
    l1 = torch.where(live, torch.logsumexp(z, 1) - z.gather(1, y.clamp(min=0).long()[:, None])[:, 0], 0.0)
    has = ids >= 0
    some = has.any(1)
    l = torch.where(has, logits.double() / tau, -float("inf"))
    l = torch.where(some[:, None], l, 0.0)
    q = torch.where(has, torch.softmax(l, 1), 0.0)
    log_p = torch.log_softmax(z / tau, 1).gather(1, ids.clamp(min=0).long())
    l2 = tau ** 2 * (torch.xlogy(q, q) - q * log_p).sum(1)
    total = (0.3 * l1.sum() + 0.7 * l2.sum()) / T
    total.backward()
    assert abs(0.3 * hard.double().sum() + 0.7 * soft.double().sum() - total * T) < 1e-5 * abs(total) * T
    dh = dh1.double() + dh2.double()
    # each gradient is off by its rounding and g's, 2^-8 of the terms: seen over the whole, a few 2^-9
    for got, want in ((dh, h64.grad), (dw1.double() + dw2.double(), w64.grad), (dz.double(), torch.where(h64 > 0, h64.grad, 0.0))):
        assert (got - want).norm() <= 4 * 2.0 ** -8 * want.norm()


def test_example_step():
    """The example's step, block and head, against 64-bit torch with autograd; what the library rounds on the
    way (y, g, dz, du and the gradients themselves) sets the tolerance: their unit roundoff, a few times over."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")
    spec = importlib.util.spec_from_file_location("expert_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for T in (6, 300):
        block, head_ = mod.ExpertBlock(136, 264, 8, 2, 4, 8, dtype=torch.float16, device=DEV, seed=T), mod.Head(136, 500, torch.float16, DEV)
        x = normal((T, 136), 1, "f16")
        y, kept = block.forward(x, torch.zeros(T, dtype=torch.int32, device=DEV))
        targets = ref.make_targets(T, 500, 2, 0.3).to(DEV)
        ids, logits = (t.to(DEV) for t in ref.make_words(T, 500, 5, 3, 0.2))
        for soft in (False, True):
            loss, dy, d_out = head_.distill(y, ids, logits, 2.0) if soft else head_.step(y, targets)
            dh, d_up, d_down = block.backward(dy, kept)
            binding.check_device_error()
            y64, out = y.double().requires_grad_(), head_.out.double().requires_grad_()
            z = y64 @ out.T
            if soft:
                has = ids >= 0
                q = torch.softmax(torch.where(has, logits.double() / 2, -1e30), 1) * has
                each = 4 * (torch.xlogy(q, q) - q * torch.log_softmax(z / 2, 1).gather(1, ids.clamp(min=0).long())).sum(1)
                n = has.any(1).sum()
            else:
                n = (targets >= 0).sum()
                each = torch.where(targets >= 0, torch.logsumexp(z, 1) - z.gather(1, targets.clamp(min=0).long()[:, None])[:, 0], 0.0)
            want = each.sum() / n
            want.backward()
            assert abs(loss.double() - want) < 1e-5 * abs(want)
            for got, grad in ((dy, y64.grad), (d_out, out.grad)):
                # (half of the smallest step per element: gradients of a mean are small numbers in binary16)
                floor = 2.0 ** -25 * got.numel() ** 0.5
                assert (got.double() - grad).norm() <= 8 * 2.0 ** -11 * grad.norm() + floor
            assert all(torch.isfinite(t.float()).all() for t in (dh, d_up, d_down)) and dh.any()


@pytest.mark.parametrize("kb", [0, 2])
def test_timed_out_wait_is_reported_and_the_next_call_is_correct(kb, monkeypatch):
    T, V, D = 50, 3000, 264
    x, w, y = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16"), ref.make_targets(T, V, 3).to(DEV)
    monkeypatch.setenv("GEMM_RELU_TEST_DROP_KB", str(kb))
    binding.gemm_relu_xent(x, w, y, b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="TIMEOUT"):
        binding.check_device_error()
    binding.check_device_error()
    for bad_T, bad_kb in ((T, 99), (300, 0)):  # no such block; pairs
        monkeypatch.setenv("GEMM_RELU_TEST_DROP_KB", str(bad_kb))
        xx = normal((bad_T, D), 1, "f16")
        with pytest.raises(binding.GemmReluError, match="INVALID"):
            binding.gemm_relu_xent(xx, w, torch.zeros(bad_T, dtype=torch.int32, device=DEV), b_layout="nk")
    monkeypatch.delenv("GEMM_RELU_TEST_DROP_KB")
    xent(x, w, y, "nk", "after the timeout")


def test_binding_refuses():
    T, V, D, k = 10, 64, 32, 3
    x, w, y = normal((T, D), 1, "f16"), head(V, D, "nk", 2, "f16"), ref.make_targets(T, V, 3).to(DEV)
    f = torch.zeros(T, device=DEV)
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, k, 4))
    for args, error in (((x.bfloat16(), w, y), TypeError), ((x.float(), w.float(), y), TypeError), ((x, w, y.long()), TypeError),
                        ((x, w, y[:-1]), ValueError), ((x, w[:, :-8], y), ValueError), ((x, w.t(), y), ValueError),
                        ((x.cpu(), w, y), ValueError), ((x, w.cpu(), y), ValueError), ((x, w, y.cpu()), ValueError),
                        ((x, w[::2], y), ValueError), ((x.t().contiguous().t(), w, y), ValueError)):
        with pytest.raises(error):
            binding.gemm_relu_xent(*args, b_layout="nk")
    with pytest.raises(ValueError):
        binding.gemm_relu_xent(x, w, y, b_layout="kv")
    with pytest.raises(binding.GemmReluError, match="ALIGNMENT"):
        binding.gemm_relu_xent(normal((T, 12), 1, "f16"), head(V, 12, "nk", 2, "f16"), y, b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="ALIGNMENT"):
        binding.gemm_relu_xent(x, head(V + 4, D, "kn", 2, "f16"), y)
    for kw, error in ((dict(loss=f.half()), TypeError), (dict(lse=f[:-1]), ValueError), (dict(loss=f.cpu()), ValueError)):
        with pytest.raises(error):
            binding.gemm_relu_xent(x, w, y, b_layout="nk", **kw)
    for lse, d, error in ((f.half(), f, TypeError), (f, f.half(), TypeError), (f, f[:-1], ValueError), (f, torch.zeros(2 * T, device=DEV)[::2], ValueError),
                          (f.cpu(), f, ValueError), (f, f.cpu(), ValueError)):
        with pytest.raises(error):
            binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout="nk")
    for kw, error in ((dict(dx=x.float()), TypeError), (dict(dx=x[:-1]), ValueError), (dict(dw=w[:-1]), ValueError), (dict(dw=w.bfloat16()), TypeError)):
        with pytest.raises(error):
            binding.gemm_relu_xent_grad(x, w, y, f, f, b_layout="nk", **kw)
    for args, error in (((ids.long(), logits), TypeError), ((ids, logits.double()), TypeError), ((ids[:, :-1], logits), ValueError),
                        ((ids[0], logits), ValueError), ((ids, logits[:-1]), ValueError), ((ids.cpu(), logits), ValueError),
                        ((ids, logits.cpu()), ValueError)):
        with pytest.raises(error):
            binding.gemm_relu_distill(x, w, *args, b_layout="nk")
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        with pytest.raises(binding.GemmReluError, match="INVALID"):
            binding.gemm_relu_distill(x, w, ids, logits, tau, b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="INVALID"):
        binding.gemm_relu_distill(x, w, ids[:, :0], logits[:, :0], b_layout="nk")
    with pytest.raises(binding.GemmReluError, match="INVALID"):
        binding.gemm_relu_distill(x, w, ids.repeat(1, 400), logits.repeat(1, 400), b_layout="nk")
    binding.check_device_error()
