"""How exact the losses over a vocabulary are, where their own rounding shows:
words that are all but certain, long reductions, small temperatures.

Every case has logits, or sums, whose error is known: either all products and
sums are exact in 32 bits (few bits each), or the tensor core's truncation is
bounded.  It cuts products and sums to 24 bits of the largest at least, so n
products of one sign and s in sum lose at most n 2^-23 s (about a sixteenth to a
tenth of that measured); a reduction in parts of n, added up in registers, at
most (n + number of parts) 2^-23 s.

Softmax, up to 256 words (E32 = 2^-23, half of it per rounding):

    s = sum 2^(c (z - max))   the maximum's own term is 1; a term of the sum goes through at most 16 additions in its
                              group of columns, 2 that join the groups, 1 from chunk to chunk, 3 from half to half and
                              3 per tile (4 at most): 34 roundings, 17 E32; twice that is allowed
    2^x                       2 units of 2^-23 and what x is off by, which is 3 roundings of it
"""
import math

import numpy as np
import pytest
import torch

import loss_ref as ref
from tiled_dense_gemm_gb300 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
BOTH = [("nk", "f16"), ("kn", "f16"), ("nk", "bf16"), ("kn", "bf16")]
E32 = ref.E32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tiled_dense_gemm_gb300 import build
    build.build()
    torch.cuda.set_device(DEV)
    yield
    torch.cuda.synchronize()


def dloss_of(T, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(T, generator=g) + 0.25).mul_(1.0 / max(T, 1)).to(DEV)


def laid_out(w, layout):
    return w if layout == "nk" else w.t().contiguous()


def exact_logits(T, V, dtype, best):
    """Rows, weights (V, 16) and their logits, of few bits each so that every sum of products is exact: word `best`
    at 40 to 104, the others 12 to 16 below it."""
    x, w = torch.zeros(T, 16), torch.zeros(V, 16)
    t, v = torch.arange(T), torch.arange(V)
    x[:, 0], x[:, 1], x[:, 2] = (40 + (t * 37) % 64).float(), ((t * 5) % 8).float() / 8, 1.0
    w[:, 0], w[:, 1], w[:, 2] = 1.0, 1.0, -(12 + ((v * 7) % 32).float() / 8)
    w[best, 2] = 0.0
    x, w = x.to(DT[dtype]), w.to(DT[dtype])
    return x.to(DEV), w.to(DEV), (x.double() @ w.double().t()).numpy()


def logsumexp(z):
    top = z.max(axis=1, keepdims=True)
    rest = np.exp(z - top)
    rest[np.arange(len(z)), z.argmax(axis=1)] = 0.0
    return top[:, 0] + np.log1p(rest.sum(axis=1)), np.log1p(rest.sum(axis=1))  # lse, lse - max


@pytest.mark.parametrize("tau", [1.0, 0.5])
@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", [1, 20, 128, 129, 300])
def test_loss_of_a_certain_word(T, layout, dtype, tau):
    """The wanted word is the maximum: its loss is the logarithm of a sum that is at least 1, so never negative, and
    off by that sum's roundings alone, however large the logits are."""
    V = 200
    for best in (0, 70, V - 1):
        x, w, z = exact_logits(T, V, dtype, best)
        lse, loss = logsumexp(z / tau)
        if tau == 1.0:
            y = torch.full((T,), best, dtype=torch.int32, device=DEV)
            got, got_lse = binding.gemm_relu_xent(x, laid_out(w, layout), y, b_layout=layout)
        else:
            ids = torch.full((T, 3), -1, dtype=torch.int32, device=DEV)
            ids[:, 1] = best
            got, got_lse = binding.gemm_relu_distill(x, laid_out(w, layout), ids, torch.zeros(T, 3, device=DEV), tau, b_layout=layout)
        binding.check_device_error()
        got, got_lse = got.double().cpu().numpy(), got_lse.double().cpu().numpy()
        e = 34 * E32
        assert (got >= 0).all(), f"{(got < 0).sum()} negative losses, least {got.min()}"
        assert (np.abs(got - tau ** 2 * loss) <= tau ** 2 * (e + 64 * E32 * loss)).all(), np.abs(got - tau ** 2 * loss).max()
        assert (np.abs(got_lse - lse) <= e + E32 * lse).all(), np.abs(got_lse - lse).max()


def check_gradients(got, g, e, x, w, layout, dtype, T, dw_steps, dx_steps, a):
    """dX and dW of g (T, V), each entry off by e before it is rounded to the type."""
    u, dt = ref.UNIT[DT[dtype]], DT[dtype]
    tiny = 2.0 ** -39 * np.abs(a).max() if dtype == "f16" else ref.TINY[dt]
    e = e + u ** (2 if T <= 32 else 1) * (np.abs(g) + e) + tiny
    n, X, W = np.abs(g) + e, x.double().cpu().numpy(), w.double().cpu().numpy()
    done = lambda v, b: (v, b + u * (np.abs(v) + b) + ref.TINY[dt])  # noqa: E731
    dx, dw = got
    ref.check(dx, done(g @ W, e @ np.abs(W) + dx_steps * E32 * (n @ np.abs(W))), "dx")
    value, bound = done(g.T @ X, e.T @ np.abs(X) + dw_steps * E32 * (n.T @ np.abs(X)))
    ref.check(dw if layout == "nk" else dw.t(), (value, bound), "dw")


@pytest.mark.parametrize("tau", [1.0, 0.5])
@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", [20, 100, 129, 300])
def test_gradient_of_a_certain_word(T, layout, dtype, tau):
    """exp(z / tau - lse) - 1 for a given lse: z and the difference are exact in 32 bits, so what is left of the
    gradient is off by the exponential's own error, not by roundings of z and lse (up to 2^-17 of 104)."""
    V, best = 200, 70
    x, w, z = exact_logits(T, V, dtype, best)
    lse = torch.from_numpy(logsumexp(z / tau)[0]).float()
    d = dloss_of(T, 3) * (256 * T)
    if tau == 1.0:
        y = torch.full((T,), best, dtype=torch.int32, device=DEV)
        got = binding.gemm_relu_xent_grad(x, laid_out(w, layout), y, lse.to(DEV), d, b_layout=layout)
    else:
        ids = torch.full((T, 2), best, dtype=torch.int32, device=DEV)
        ids[:, 1] = -1
        got = binding.gemm_relu_distill_grad(x, laid_out(w, layout), ids, torch.zeros(T, 2, device=DEV), lse.to(DEV), d, tau, b_layout=layout)
    binding.check_device_error()
    arg = z / tau - lse.double().numpy()[:, None]
    p, a = np.exp(arg), d.double().cpu().numpy()[:, None] * tau
    g = p.copy()
    g[:, best] = np.expm1(arg[:, best])
    # (two roundings of the factor, one each of the product and the difference)
    e = np.abs(a) * (p * (2 + 3 * np.abs(arg) + 2) * E32)
    e[:, best] += np.abs(a)[:, 0] * 2 * E32
    check_gradients(got, a * g, e, x, w, layout, dtype, T, T, V + 32, a)


def nearly_certain(T, D, V, dtype, seed, size=24.0):
    """Rows along the weights of a word each, whose logit is about `size`; another word's is half of that.  All
    products of the largest logits have one sign, where truncation takes most."""
    gen = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=gen) * 2 * D ** -0.5).to(DT[dtype])
    half = V // 2
    w[half:] = (0.5 * w[:half].float()).to(DT[dtype])
    y = torch.randint(0, half, (T,), generator=gen, dtype=torch.int32)
    rows = w[y.long()].float()
    lift = size + 8 * torch.rand(T, 1, generator=gen)
    x = (lift * rows / rows.pow(2).sum(dim=1, keepdim=True)).to(DT[dtype])
    return x.to(DEV), w.to(DEV), y.to(DEV)


def truncated(T, x, w, parts_of):
    """What z may be off by, z summed in parts of so many products."""
    D = x.shape[1]
    size = x.double().cpu().numpy(), w.double().cpu().numpy()
    return np.abs(size[0]) @ np.abs(size[1]).T * E32 * (min(D, parts_of) + math.ceil(D / parts_of))


@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", [1, 20, 128])
def test_lse_of_up_to_128_rows_with_a_certain_word(T, layout, dtype):
    """The logit of the wanted word is summed exactly (2048 products in 256 threads' numbers), so lse is off by its
    own rounding, the sum's, and what truncation makes of the words that have little part in it."""
    V, D = 64, 2048
    x, w, y = nearly_certain(T, D, V, dtype, T)
    z = x.double().cpu().numpy() @ w.double().cpu().numpy().T
    lse, loss = logsumexp(z)
    small = 2 * truncated(T, x, w, 256).max(axis=1) * loss
    got, got_lse = binding.gemm_relu_xent(x, laid_out(w, layout), y, b_layout=layout)
    binding.check_device_error()
    off, off_lse = np.abs(got.double().cpu().numpy() - loss), np.abs(got_lse.double().cpu().numpy() - lse)
    # (64 words are one chunk: 16 additions, 2 that join, 1, 3 and 3)
    e = 25 * E32 / 2 + small + 4 * E32 * loss
    assert (off_lse <= e + E32 / 2 * lse).all(), (off_lse / lse).max()
    assert (off <= e).all(), off.max()
    for tau in (1.0, 1.5):
        # q in two places of the same word, and a little elsewhere
        ids = torch.stack([y, y, (y + 1) % V, torch.full_like(y, -1)], dim=1).contiguous()
        logits = torch.tensor([9.0, 9.5, -9.0, 50.0], device=DEV).expand(T, 4).contiguous()
        lse = logsumexp(z / tau)[0]
        _, got_lse = binding.gemm_relu_distill(x, laid_out(w, layout), ids, logits, tau, b_layout=layout)
        binding.check_device_error()
        rest = logsumexp(z / tau)[1]
        e = 25 * E32 / 2 + 2 * truncated(T, x, w, 256).max(axis=1) / tau * rest + 4 * E32 * rest + E32 / 2 * lse
        off_lse = np.abs(got_lse.double().cpu().numpy() - lse)
        assert (off_lse <= e).all(), (off_lse / lse).max()


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("D", [8, 72, 264, 1000, 8200, 40008])
@pytest.mark.parametrize("T", [1, 7, 128])
def test_lse_of_certain_words_of_any_width(T, D, layout):
    """The exact logits are summed in shares over warps and CTAs, as many as the width and the rows give."""
    V = 64
    x, w, y = nearly_certain(T, D, V, "f16", T + D)
    z = x.double().cpu().numpy() @ w.double().cpu().numpy().T
    best, (lse, loss) = z.argmax(axis=1), logsumexp(z)
    ok = loss < 0.6  # (p > 1/2: 8 numbers at random may lie closer than the words' halves)
    got, got_lse = binding.gemm_relu_xent(x, laid_out(w, layout), torch.from_numpy(best).int().to(DEV), b_layout=layout)
    binding.check_device_error()
    e = 25 * E32 / 2 + 2 * truncated(T, x, w, 256).max(axis=1) * loss + 4 * E32 * loss
    off, off_lse = np.abs(got.double().cpu().numpy() - loss), np.abs(got_lse.double().cpu().numpy() - lse)
    assert ok.any()
    assert (off_lse <= e + E32 / 2 * lse)[ok].all(), (off_lse / lse)[ok].max()
    assert (off <= e)[ok].all(), off[ok].max()


@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T,D", [(1, 2048), (20, 2048), (100, 2048), (129, 2056), (300, 4096), (300, 1544)])
def test_gradients_of_certain_words_with_the_forward_pass_own_lse(T, D, layout, dtype):
    """The true gradient, with lse as the forward call returned it: both passes sum a logit alike (or exactly), so
    what the tensor core truncates of it takes the same part of 1 - p, not of p."""
    V = 64
    x, w, y = nearly_certain(T, D, V, dtype, T + D)
    z = x.double().cpu().numpy() @ w.double().cpu().numpy().T
    lse, loss = logsumexp(z)
    d = dloss_of(T, 3) * (256 * T)
    _, got_lse = binding.gemm_relu_xent(x, laid_out(w, layout), y, b_layout=layout)
    got = binding.gemm_relu_xent_grad(x, laid_out(w, layout), y, got_lse, d, b_layout=layout)
    binding.check_device_error()
    at, a = (np.arange(T), y.cpu().numpy()), d.double().cpu().numpy()[:, None]
    p = np.exp(z - lse[:, None])
    g, rest = p.copy(), -np.expm1(-loss)  # 1 - p of the wanted word
    g[at] = -rest
    b = truncated(T, x, w, 256 if T <= 128 else 1024).max(axis=1)
    arg = np.abs(z - lse[:, None])
    # lse: its own rounding and its sum's; the exponential's argument and value
    shift = E32 / 2 * lse + 25 * E32 / 2
    e = p * (2 * b[:, None] + shift[:, None] + (4 + 3 * arg) * E32)
    e[at] = rest * 2 * b + shift + 8 * E32
    check_gradients(got, a * g, a * e, x, w, layout, dtype, T, T, V + 32, a)


@pytest.mark.parametrize("ignored", [0.0, 0.4])
@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("D", [1032, 2056, 4096])
@pytest.mark.parametrize("T", [100, 129, 300, 513])
def test_reductions_in_parts(T, D, layout, dtype, ignored):
    """Logits of spread 2 over widths that are summed in several parts: within the bounds row by row, and over all
    rows as exact as the parts make them.  Sixteen products at a time lose up to a unit of 2^-23 of the sum so far, low: over n about
    n / 16 * 2^-23 of its size, which for a spread of 2 is about 4, a third of the loss.  Parts of 256 (up to 128
    rows): 3e-7 would take 7 of such steps' units; of 1024: 1e-6; one part of 4096 measured 2.4e-6."""
    V = 1000
    gen = torch.Generator(device=DEV).manual_seed(D + T)
    x = torch.randn((T, D), generator=gen, device=DEV).to(DT[dtype])
    w = (torch.randn((V, D), generator=gen, device=DEV) * 2 * D ** -0.5).to(DT[dtype])
    y = ref.make_targets(T, V, T, ignored).to(DEV)
    y[0] = 1
    valid = y >= 0
    z = x.double() @ w.double().t()
    lse = torch.where(valid, torch.logsumexp(z, 1), 0.0)
    loss = torch.where(valid, lse - z.gather(1, y.clamp(min=0).long()[:, None])[:, 0], 0.0)
    got, got_lse = binding.gemm_relu_xent(x, laid_out(w, layout), y, b_layout=layout)
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, 7, T, ignored))
    soft, soft_lse = binding.gemm_relu_distill(x, laid_out(w, layout), ids, logits, 2.0, b_layout=layout)
    binding.check_device_error()
    rms = 3e-7 if T <= 128 else 1e-6
    rel = ((got_lse.double() - lse)[valid] / lse[valid]).pow(2).mean().sqrt().item()
    assert rel <= rms, rel
    off = ((got.double() - loss)[valid].pow(2).mean() / loss[valid].pow(2).mean()).sqrt().item()
    assert off <= rms, off
    assert not got[~valid].any() and not got_lse[~valid].any()
    has = (ids >= 0).any(1)
    lse2 = torch.logsumexp(z / 2, 1)
    rel = ((soft_lse.double() - lse2)[has] / lse2[has]).pow(2).mean().sqrt().item()
    assert rel <= rms, rel
    want, _ = ref.losses(x, laid_out(w, layout), ref.words_of(ids=ids, logits=logits, tau=2.0), layout, 2.0, False)
    ref.check(soft, want, "distill")
    # the gradients' z in the same parts
    d = dloss_of(T, 5)
    dx, dw = binding.gemm_relu_xent_grad(x, laid_out(w, layout), y, got_lse, d, b_layout=layout)
    binding.check_device_error()
    rx, rw = ref.gradients(x, laid_out(w, layout), ref.words_of(targets=y), got_lse, d, layout)
    ref.check(dx, rx, "dx")
    ref.check(dw, rw, "dw")


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("ignored", [False, True])
def test_weight_gradient_of_many_rows(layout, ignored):
    """Sums over a million rows of terms of one sign: of two words with a logit of 0 and six far below, g is +-a / 2
    exactly, and the rows are positive: in one accumulator the sum lost 1.07% of itself.  In parts of 4096 rows it
    loses at most 2^-23 * (4096 + 256), beside its own rounding."""
    T, V, D = 1 << 20, 8, 64
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = (torch.randint(64, 128, (T, D), generator=gen, device=DEV).float() / 128).half()
    x[:, D - 1] = 1.0
    w = torch.zeros((V, D), dtype=torch.float16, device=DEV)
    w[2:, D - 1] = -200.0
    y = torch.zeros(T, dtype=torch.int32, device=DEV)
    if ignored:
        y[torch.rand(T, generator=gen, device=DEV) < 0.3] = -1
    a = torch.full((1,), 2.0 ** -20, device=DEV)
    loss, lse = binding.gemm_relu_xent(x, laid_out(w, layout), y, b_layout=layout)
    dx, dw = binding.gemm_relu_xent_grad(x, laid_out(w, layout), y, lse, a, b_layout=layout)
    binding.check_device_error()
    total = 2.0 ** -21 * x[y >= 0].double().sum(0)
    dw = dw if layout == "nk" else dw.t()
    bound = total * (2.0 ** -11 + 1.001 * (4096 + T / 4096) * E32)
    for row, want in ((0, -total), (1, total)):
        off = (dw[row].double() - want).abs()
        assert (off <= bound).all(), (off / total).max().item()
    assert not dw[2:].any() and not dx[:, :-1].any()


@pytest.mark.parametrize("T,V", [(1, 16000000), (100, 4200008), (200, 2200008)])
def test_row_gradient_of_many_words(T, V):
    """Sums over millions of words of terms of one sign: the words' logits are 0, so g is a / V at every word but the
    target (G's own rounding is the same at all of them), and their weights are positive.  In one accumulator per
    share dX lost 0.2%; in parts of 4096 words it loses at most 2^-23 * (4096 + V / 4096)."""
    D = 16
    gen = torch.Generator(device=DEV).manual_seed(6)
    w = (torch.randint(64, 128, (V, D), generator=gen, device=DEV).float() / 128).half()
    x = torch.zeros((T, D), dtype=torch.float16, device=DEV)
    y = torch.zeros(T, dtype=torch.int32, device=DEV)
    w[0] = 0
    lse = torch.full((T,), math.log(V), device=DEV)
    d = torch.full((T,), 1.0, device=DEV)
    dx, _ = binding.gemm_relu_xent_grad(x, w, y, lse, d, want_dw=False, b_layout="nk")
    binding.check_device_error()
    p = math.exp(-lse[0].double().item())
    # G is p times 2047 / 1024 * 2^14, rounded (twice up to 32 rows: to its rest's half unit)
    scale = 2047.0 / 1024.0 * 2 ** 14
    g = torch.tensor(p * scale, dtype=torch.float64)
    held = g.half().double()
    if T <= 32:
        held = held + (g - held).half().double()
    want = w.double().sum(0) * held / scale
    # the exponential: 2 units, its argument of 16.6 three roundings, the factor two; a step of G (of its rest: 2^-24)
    # more where that crosses a border of its rounding
    e, step = (4 + 3 * 16.6) * E32, 2.0 ** (math.floor(math.log2(g.item())) - 10)
    if T <= 32:
        unit = 2.0 ** -24 / g.item()
    else:
        unit = step / g.item() if abs((g - held).item()) > step / 2 - 2 * e * g.item() else 0.0
    bound = want * (e + unit + 2.0 ** -11 + 1.001 * (4096 + V / 4096) * E32)
    off = (dx.double() - want).abs()
    assert (off <= bound).all(), (off / want).max().item()


@pytest.mark.parametrize("T,V,k", [(2100, 140003, 5), (31, 4200008, 3), (128, 2200008, 3)])
def test_several_pieces_with_a_teacher(T, V, k):
    """A teacher's words in every piece of the vocabulary, at both sides of the pieces' borders, some certain."""
    D, tau = 16, 2.0
    gen = torch.Generator(device=DEV).manual_seed(7)
    w = (torch.randn((V, D), generator=gen, device=DEV) * 2 * D ** -0.5).bfloat16()
    x = torch.randn((T, D), generator=gen, device=DEV).bfloat16()
    ids = torch.randint(0, V, (T, k), generator=gen, device=DEV, dtype=torch.int32)
    rows = max(T, 1) if T > 32 else 2 * ((T + 7) // 8 * 8)
    most = max(256, (1 << 29) // (2 * rows) // 256 * 256)
    piece = -(-(-(-V // -(-V // most))) // 256) * 256
    assert piece < V
    edge = torch.tensor([piece - 1, piece, 0, V - 1], device=DEV, dtype=torch.int32)
    ids[:, 0] = edge[torch.arange(T, device=DEV) % 4]
    ids[::5, 1] = -1
    ids[3::7] = -1
    sure = torch.arange(T, device=DEV) % 3 == 1
    word = w[ids[:, 0].clamp(min=0).long()].float()
    x[sure] = (60 * word / word.pow(2).sum(dim=1, keepdim=True)).to(x.dtype)[sure]
    logits = torch.randn((T, k), generator=gen, device=DEV)
    logits[sure, 0] = 12.0
    d = dloss_of(T, 8)
    has = ids >= 0
    live = has.any(1)
    q = torch.softmax(torch.where(has, logits.double() / tau, -1e30), 1) * has
    lse = torch.zeros(T, device=DEV)
    rows = torch.arange(T, device=DEV)
    u = 2.0 ** -8
    W, X = w.double(), torch.where(live[:, None], x.double(), 0.0)
    dx, ex = torch.zeros((T, D), dtype=torch.float64, device=DEV), torch.zeros((T, D), dtype=torch.float64, device=DEV)
    dw, ew = torch.zeros((V, D), dtype=torch.float64, device=DEV), torch.zeros((V, D), dtype=torch.float64, device=DEV)
    for at in rows.split(256):
        z = x[at].double() @ W.t() / tau
        lse[at] = torch.where(live[at], torch.logsumexp(z, 1), 0.0).float()
        a = (torch.where(live[at], d[at], torch.zeros(()).to(DEV)) * tau).double()[:, None]
        r = lse[at].double()[:, None]
        p = torch.exp(z - r)
        ez = D * E32 * (x[at].double().abs() @ W.abs().t()) / tau
        e = p * (ez + 2 * E32 * (z.abs() + r.abs()) + 2 * E32)
        here = torch.arange(len(at), device=DEV)
        # (a row's first word, of p above a half, from a sum in 64 bits)
        top = ids[at, 0].clamp(min=0).long()
        if T <= 128:
            exact = p[here, top] * (ez[here, top] / D + 2 * E32)
            e[here, top] = torch.where((p[here, top] > 0.501) & has[at, 0], exact, e[here, top])
        size = p.clone()
        for j in range(k):
            i = ids[at, j].clamp(min=0).long()
            p.index_put_((here, i), -q[at, j], accumulate=True)
            size.index_put_((here, i), q[at, j], accumulate=True)
            e.index_put_((here, i), q[at, j] * (40 + k) * E32, accumulate=True)
        g, e = a * p, a * (e + 4 * E32 * size)
        e = e + u ** (2 if T <= 32 else 1) * (g.abs() + e) + (2.0 ** -134) * live[at].double()[:, None]
        n = g.abs() + e
        dx[at], ex[at] = g @ W, e @ W.abs() + V / 16 * E32 * (n @ W.abs())
        dw += g.t() @ X[at]
        ew += e.t() @ X[at].abs() + T * E32 * (n.t() @ X[at].abs())
        del z, p, ez, e, size, g, n
    got_dx, got_dw = binding.gemm_relu_distill_grad(x, w, ids, logits, lse, d, tau, b_layout="nk")
    binding.check_device_error()
    for out, value, bound in ((got_dw, dw, ew), (got_dx, dx, ex)):
        off = (out.double() - value).abs() - (bound + u * (value.abs() + bound) + 2.0 ** -134)
        assert off.max().item() <= 0.0
    assert not got_dx[~live].any()


@pytest.mark.parametrize("layout,dtype", BOTH)
@pytest.mark.parametrize("T", [7, 32, 90, 300])
def test_gradients_of_losses_of_both_signs_and_many_sizes(T, layout, dtype):
    """dloss below zero, of both signs among the rows, and over eleven orders of magnitude: binary16's G keeps
    2^-29 of the largest in full and loses what is below 2^-40 of it."""
    V, D, k, tau = 504, 136, 4, 1.5
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, D, generator=gen).to(DT[dtype]).to(DEV)
    w = laid_out((torch.randn(V, D, generator=gen) * 2 * D ** -0.5).to(DT[dtype]).to(DEV), layout)
    y = ref.make_targets(T, V, T, 0.2).to(DEV)
    ids, logits = (t.to(DEV) for t in ref.make_words(T, V, k, T + 1, 0.2))
    base = dloss_of(T, T + 2)
    sign = torch.where(torch.arange(T, device=DEV) % 3 == 0, -1.0, 1.0)
    size = 10.0 ** -(torch.arange(T, device=DEV) % 12).float()
    _, lse = binding.gemm_relu_xent(x, w, y, b_layout=layout)
    _, soft = binding.gemm_relu_distill(x, w, ids, logits, tau, b_layout=layout)
    for d in (-base, base * sign, base * sign * size, torch.full((1,), -0.01, device=DEV)):
        got = binding.gemm_relu_xent_grad(x, w, y, lse, d, b_layout=layout)
        want = ref.gradients(x, w, ref.words_of(targets=y), lse, d, layout)
        for name, o, r in zip(("dx", "dw"), got, want):
            ref.check(o, r, name)
        got = binding.gemm_relu_distill_grad(x, w, ids, logits, soft, d, tau, b_layout=layout)
        want = ref.gradients(x, w, ref.words_of(ids=ids, logits=logits, tau=tau), soft, d, layout, tau, cross=False)
        for name, o, r in zip(("dx", "dw"), got, want):
            ref.check(o, r, f"{name} with a teacher")
    binding.check_device_error()


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("T", [20, 100])
def test_gradient_of_a_main_word_in_several_entries(T, layout):
    """A word whose weight of 0.6 comes in four entries of 0.15 beside one of 0.4: it is the row's main word all the
    same, so p - q there, next to nothing, comes from the exact sum of z."""
    V, D, tau = 64, 2048, 1.0
    gen = torch.Generator().manual_seed(T)
    w = (torch.randn(V, D, generator=gen) * 2 * D ** -0.5).half()
    a, b = w[3].float(), w[40].float()
    pair = torch.stack([a, b])
    for_both = torch.linalg.solve((pair @ pair.t()).double(), torch.tensor([1.0, 1.0], dtype=torch.float64))
    only_a = torch.linalg.solve((pair @ pair.t()).double(), torch.tensor([1.0, 0.0], dtype=torch.float64))
    both, first = (for_both @ pair.double()), (only_a @ pair.double())
    x = ((20 + 8 * torch.rand(T, 1, generator=gen)).double() * both + math.log(1.5) * first).half()
    ids = torch.tensor([3, 40, 3, 3, 3], dtype=torch.int32).repeat(T, 1).to(DEV)
    logits = torch.log(torch.tensor([0.15, 0.4, 0.15, 0.15, 0.15])).repeat(T, 1).to(DEV)
    q = 4 * torch.softmax(logits[0].double(), 0)[0].item()
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1).float()
    d = dloss_of(T, 3) * (256 * T)
    _, dw = binding.gemm_relu_distill_grad(x.to(DEV), laid_out(w.to(DEV), layout), ids, logits, lse.to(DEV), d, tau, b_layout=layout)
    binding.check_device_error()
    p = torch.exp(z[:, 3] - lse.double())
    s = d.double().cpu()
    g = s * (p - q)
    # the exponential and the argument's rounding; four weights, their logits' and the softmax's roundings
    e = s * (8 * E32 + q * (4 * 2 + 8 + 5 + 4) * E32)
    e = e + 2.0 ** (-22 if T <= 32 else -11) * (g.abs() + e) + 2.0 ** -39 * s.max()
    value, bound = x.double().t() @ g, x.double().abs().t() @ e + T * E32 * (x.double().abs().t() @ (g.abs() + e))
    bound += 2.0 ** -11 * (value.abs() + bound) + 2.0 ** -25
    off = ((dw[3] if layout == "nk" else dw[:, 3]).double().cpu() - value).abs()
    assert (off <= bound).all(), ((off / bound).max().item(), (p - q).abs().max().item())


@pytest.mark.parametrize("tau", [2.0 ** -20, 2.0 ** -70, 1e-22])
@pytest.mark.parametrize("T", [20, 300])
def test_small_temperatures(T, tau):
    """tau^2 may leave 32 bits where tau times the gap between the logits does not."""
    V, best, word = 200, 70, 3
    tau = float(np.float32(tau))
    x, w, z = exact_logits(T, V, "f16", best)
    ids = torch.full((T, 1), word, dtype=torch.int32, device=DEV)
    loss, lse = binding.gemm_relu_distill(x, w, ids, torch.zeros(T, 1, device=DEV), tau, b_layout="nk")
    binding.check_device_error()
    want = tau * (z[:, best] - z[:, word])
    assert (np.abs(loss.double().cpu().numpy() - want) <= 4 * E32 * want).all()
    assert (np.abs(lse.double().cpu().numpy() - z[:, best] / tau) <= 4 * E32 * z[:, best] / tau).all()
