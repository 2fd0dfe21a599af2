"""Cases and plain forms of the ragged products: rows of one batch that go
through different weights.

Four operators of the package are measured here:

* ``grouped``     y[t] = ReLU(x[t] @ w[g(t)])           (experts' products)
* ``grouped_dx``  dx[t] = (dy[t] @ w[g(t)]^T) * (act[t] > 0)
* ``grouped_dw``  dw[g] = x[rows of g]^T @ dy[rows of g]
* ``adapters``    y[t] = ReLU(x[t] @ w + scale[i] * (x[t] @ a[i]^T) @ b[i]),
                  i = ids[t] (no adapter where ids[t] is -1)

Rows are sorted by group; ``offsets`` (device, int32) holds each group's first
row and the end of the last one.  A row of no group gets zeros.
"""
import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    """The cases; see the comment at each for what it stands for."""
    return [
        # four tokens with two experts each, in a buffer with room for more:
        # one step of a small decode, where latency counts
        dict(name="grouped decode 8 rows", op="grouped", dtype="f16", layout="kn", relu=True, T=16, used=8, G=16, active=6, K=1024, N=1024, skew=0.5),
        # a decode batch that reaches every one of 64 experts with a few rows:
        # the experts' weights are what is read
        dict(name="grouped decode 256 rows", op="grouped", dtype="bf16", layout="kn", relu=False, T=256, used=256, G=64, active=64, K=4096, N=2048, skew=0.5),
        # the up projection of a training step or a long prompt, uneven routing
        dict(name="grouped up 16384 rows", op="grouped", dtype="bf16", layout="kn", relu=True, T=16384, used=16384, G=32, active=32, K=2048, N=4096, skew=0.5),
        # sizes that divide nothing, weights stored (N, K), some experts empty
        dict(name="grouped ragged 5000 rows", op="grouped", dtype="f16", layout="nk", relu=True, T=5000, used=4987, G=12, active=9, K=2056, N=3000, skew=1.0),
        # the data gradient of that up projection's successor, with the ReLU's
        # gradient of the activations it was given
        dict(name="grouped_dx 16384 rows", op="grouped_dx", dtype="bf16", layout="kn", act=True, T=16384, used=16384, G=32, active=32, K=2048, N=4096, skew=0.5),
        # a small fine-tuning step, no ReLU below, odd sizes
        dict(name="grouped_dx 300 rows", op="grouped_dx", dtype="f16", layout="kn", act=False, T=300, used=300, G=16, active=13, K=1000, N=520, skew=1.0),
        # a middle-sized step with weights stored (N, K)
        dict(name="grouped_dx 3000 rows", op="grouped_dx", dtype="bf16", layout="nk", act=True, T=3000, used=3000, G=8, active=8, K=1024, N=4096, skew=0.5),
        # the weight gradient of the training step
        dict(name="grouped_dw 16384 rows", op="grouped_dw", dtype="bf16", layout="kn", T=16384, used=16384, G=32, active=32, K=2048, N=4096, skew=0.5),
        # short ragged groups, some without a row: the gradients written are
        # most of the work
        dict(name="grouped_dw 1000 rows", op="grouped_dw", dtype="f16", layout="kn", T=1000, used=1000, G=24, active=20, K=1032, N=520, skew=1.0),
        # one token of one request
        dict(name="adapters 1 row", op="adapters", dtype="f16", layout="kn", relu=True, T=1, K=4096, N=4096, R=8, used=1, rank=16, segments=0),
        # a decode batch of 64 requests, each with its adapter or none
        dict(name="adapters decode 64 rows", op="adapters", dtype="bf16", layout="kn", relu=False, T=64, K=8192, N=8192, R=64, used=48, rank=32, segments=0),
        # prompts of a few requests beside decoding ones, in one batch
        dict(name="adapters prompts 8192 rows", op="adapters", dtype="bf16", layout="kn", relu=True, T=8192, K=4096, N=4096, R=32, used=24, rank=64, segments=40),
    ]


def _log_int(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))


def _dim(rng, lo, hi):
    """A width: a multiple of 8, as the rows' 16-byte pitch asks; half of them are multiples of 64."""
    unit = rng.choice((8, 64))
    return max(unit, _log_int(rng, lo, hi) // unit * unit)


def draw(rng):
    """One more case of the listed ones' ranges, no larger than their largest."""
    op = rng.choice(("grouped", "grouped", "grouped_dx", "grouped_dw", "adapters"))
    case = dict(op=op, dtype=rng.choice(("f16", "bf16")), layout=rng.choice(("kn", "kn", "nk")))
    k, n = _dim(rng, 256, 8192), _dim(rng, 256, 8192)
    t = _log_int(rng, 1, 16384)
    t = max(1, min(t, 130_000_000_000 // (k * n)))
    if op == "adapters":
        r = _log_int(rng, 1, 64)
        rank = rng.choice((4, 8, 16, 16, 20, 32, 64))
        segments = 0 if t <= 256 else rng.randint(1, min(t, 64))
        used = rng.randint(1, max(1, min(r, segments or t)))
        case.update(relu=rng.random() < 0.5, T=t, K=k, N=n, R=r, used=used, rank=rank, segments=segments)
        return case
    g = min(_log_int(rng, 1, 128), 500_000_000 // (k * n))
    used = t if rng.random() < 0.7 else rng.randint(1, t)
    active = rng.randint(max(1, min(g, used) // 2), min(g, used))
    case.update(T=t, used=used, G=g, active=active, K=k, N=n, skew=rng.choice((0.0, 0.5, 1.0)))
    if op == "grouped":
        case["relu"] = rng.random() < 0.5
    elif op == "grouped_dx":
        case["act"] = rng.random() < 0.5
    return case


def _group_sizes(case, rs):
    """Rows of each group: `active` groups have at least one, the rest go by uneven odds."""
    g, active = case["G"], case["active"]
    odds = np.zeros(g)
    chosen = rs.permutation(g)[:active]
    odds[chosen] = np.exp(case["skew"] * rs.standard_normal(active))
    sizes = np.zeros(g, dtype=np.int64)
    sizes[chosen] = 1
    return sizes + rs.multinomial(case["used"] - active, odds / odds.sum())


def _adapter_ids(case, rs):
    """Each row's adapter: `used` of them occur; about one request in ten has none."""
    t, used, segments = case["T"], case["used"], case["segments"]
    requests = segments or t
    chosen = rs.permutation(case["R"])[:used]
    of = np.concatenate([chosen, rs.choice(chosen, requests - used)])
    of[used:][rs.random_sample(requests - used) < 0.1] = -1
    of = of[rs.permutation(requests)]
    if not segments:
        return of.astype(np.int32)
    # prompts of uneven length, one row at least (a decoding request)
    lengths = 1 + rs.multinomial(t - segments, rs.dirichlet(np.full(segments, 0.5)))
    return np.repeat(of, lengths).astype(np.int32)


def prepare(case, seed):
    """Inputs on the GPU: activations of order one, weights that keep them so, gradients of order one."""
    dtype, dev = DTYPES[case["dtype"]], "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (2 ** 32 - 1))

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    op, t, k, n = case["op"], case["T"], case["K"], case["N"]
    state = dict(op=op, layout=case["layout"])
    if op == "adapters":
        rank, r = case["rank"], case["R"]
        w = normal(*((k, n) if case["layout"] == "kn" else (n, k)), scale=k ** -0.5)
        state.update(relu=case["relu"], x=normal(t, k), w=w, a=normal(r, rank, k, scale=k ** -0.5), b=normal(r, rank, n, scale=rank ** -0.5),
                     ids=torch.from_numpy(_adapter_ids(case, rs)).to(dev),
                     scale=torch.rand(r, generator=gen, device=dev, dtype=torch.float32) + 0.5)
        return state
    sizes = _group_sizes(case, rs)
    ends = np.cumsum(sizes)
    state["offsets"] = torch.from_numpy(np.concatenate([[0], ends]).astype(np.int32)).to(dev)
    state["most"] = int(sizes.max())  # rows of the largest group, for the plain form's padded product
    if op != "grouped_dw":
        state["w"] = normal(case["G"], *((k, n) if case["layout"] == "kn" else (n, k)), scale=(k if op == "grouped" else n) ** -0.5)
    if op == "grouped":
        state.update(relu=case["relu"], x=normal(t, k))
    elif op == "grouped_dx":
        state.update(dy=normal(t, n), act=torch.relu(normal(t, k)) if case["act"] else None)
    else:
        state.update(x=normal(t, k), dy=normal(t, n))
    return state


def _places(offsets, most, t):
    """Of the padded (group, place) grid: each place's row and whether it is one; of the rows: their group, place and whether they have one."""
    start, end = offsets[:-1].long(), offsets[1:].long()
    row = start[:, None] + torch.arange(most, device=offsets.device)
    real = row < end[:, None]
    rows = torch.arange(t, device=offsets.device)
    group = torch.searchsorted(end, rows, right=True)
    inside = group < end.numel()
    group = group.clamp(max=end.numel() - 1)
    place = (rows - start[group]).clamp(0, most - 1)
    return row.clamp(max=t - 1), real, group, place, inside


def _plain(s):
    op = s["op"]
    if op == "adapters":
        x, ids = s["x"].float(), s["ids"].long()
        w = s["w"].float() if s["layout"] == "kn" else s["w"].float().t()
        has = ids >= 0
        every = torch.einsum("tk,rjk->trj", x, s["a"].float())  # every adapter's low-rank part of every row
        mine = torch.nn.functional.one_hot(ids.clamp(min=0), s["a"].shape[0]) * has[:, None]
        every = every * (mine * s["scale"])[:, :, None]
        y = x @ w + every.flatten(1) @ s["b"].float().flatten(0, 1)
        return (torch.relu(y) if s["relu"] else y).to(s["x"].dtype)
    first = s["dy"] if op == "grouped_dx" else s["x"]
    row, real, group, place, inside = _places(s["offsets"], s["most"], first.shape[0])
    padded = first.float()[row] * real[:, :, None]
    if op == "grouped_dw":
        dy = s["dy"].float()[row] * real[:, :, None]
        dw = padded.transpose(1, 2) @ dy
        return (dw if s["layout"] == "kn" else dw.transpose(1, 2)).to(first.dtype).contiguous()
    w = s["w"].float()
    if (s["layout"] == "nk") == (op == "grouped"):
        w = w.transpose(1, 2)
    y = (padded @ w)[group, place] * inside[:, None]
    if op == "grouped":
        return (torch.relu(y) if s["relu"] else y).to(first.dtype)
    return (y if s["act"] is None else y * (s["act"] > 0)).to(first.dtype)


def run(state):
    """One pass through one operator."""
    if not own:
        return _plain(state)
    import tiled_dense_gemm_gb300 as fw
    op = state["op"]
    if op == "grouped":
        return fw.gemm_relu_grouped(state["x"], state["w"], state["offsets"], apply_relu=state["relu"], b_layout=state["layout"])
    if op == "grouped_dx":
        return fw.gemm_relu_grouped_dx(state["dy"], state["w"], state["offsets"], act=state["act"], b_layout=state["layout"])
    if op == "grouped_dw":
        return fw.gemm_relu_grouped_dw(state["x"], state["dy"], state["offsets"], b_layout=state["layout"])
    return fw.gemm_relu_adapters(state["x"], state["w"], state["a"], state["b"], state["ids"], state["scale"],
                                 apply_relu=state["relu"], b_layout=state["layout"])


def work(case):
    """Bytes and operations that one pass cannot do without: the rows in use, the weights they reach, every output."""
    k, n, t, used = case["K"], case["N"], case["T"], case["used"]
    if case["op"] == "adapters":
        r = case["rank"]
        rows = 2 * t * (k + n) + 4 * t
        return {"bytes": rows + 2 * k * n + used * (2 * r * (k + n) + 4), "flops": 2 * t * (k * n + r * (k + n))}
    g, active = case["G"], case["active"]
    flops = 2 * used * k * n
    if case["op"] == "grouped":
        return {"bytes": 2 * (used * k + t * n + active * k * n) + 4 * (g + 1), "flops": flops}
    if case["op"] == "grouped_dx":
        act = used * k if case["act"] else 0
        return {"bytes": 2 * (used * n + t * k + act + active * k * n) + 4 * (g + 1), "flops": flops}
    return {"bytes": 2 * (used * (k + n) + g * k * n) + 4 * (g + 1), "flops": flops}


def exact(case, seed):
    """The same outputs in 64 bits, group by group and adapter by adapter from the definitions."""
    s = prepare(case, seed)
    op, nk = case["op"], case["layout"] == "nk"
    if op == "adapters":
        x, w = s["x"].double(), s["w"].double()
        y = torch.matmul(x, w.T if nk else w)
        ids = s["ids"].cpu().numpy()
        for i in sorted(set(ids.tolist()) - {-1}):
            at = torch.from_numpy(np.flatnonzero(ids == i)).to(x.device)
            low = torch.matmul(x[at], s["a"][i].double().T)
            y[at] += float(s["scale"][i]) * torch.matmul(low, s["b"][i].double())
        return y.clamp(min=0) if case["relu"] else y
    bounds = s["offsets"].cpu().tolist()
    k, n = case["K"], case["N"]
    if op == "grouped_dw":
        out = torch.zeros((case["G"], n, k) if nk else (case["G"], k, n), dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros((case["T"], n if op == "grouped" else k), dtype=torch.float64, device="cuda")
    for g, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        if lo == hi:
            continue
        if op == "grouped_dw":
            x, dy = s["x"][lo:hi].double(), s["dy"][lo:hi].double()
            out[g] = torch.matmul(dy.T, x) if nk else torch.matmul(x.T, dy)
            continue
        w = s["w"][g].double()
        if op == "grouped":
            y = torch.matmul(s["x"][lo:hi].double(), w.T if nk else w)
            out[lo:hi] = y.clamp(min=0) if case["relu"] else y
        else:
            d = torch.matmul(s["dy"][lo:hi].double(), w if nk else w.T)
            out[lo:hi] = d if s["act"] is None else torch.where(s["act"][lo:hi] > 0, d, torch.zeros_like(d))
    return out
