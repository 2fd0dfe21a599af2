"""Cases and plain forms of the losses over a vocabulary: the product of a
model's last rows with its output weights, the softmax over the whole
vocabulary and what is left of it (a loss per row, the gradients), with no
logits kept.

Four operators of the package are measured here, z[t] = x[t] @ w (one logit
per word; w is (D, V), or (V, D) for layout "nk"):

* ``xent``          lse[t] = log sum_v exp z[t, v],  loss[t] = lse[t] - z[t, y(t)]
* ``xent_grad``     g[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - [v = y(t)]),
                    dx = g @ w^T,  dw = x^T @ g (laid out as w)
* ``distill``       the teacher's k best words of each row, ids and logits, tau a temperature:
                    q = softmax of those logits / tau,  lse[t] = log sum_v exp(z[t, v] / tau),
                    loss[t] = tau^2 sum_j q_j (log q_j - z[t, id_j] / tau + lse[t])
* ``distill_grad``  g[t, v] = dloss[t] tau (exp(z[t, v] / tau - lse[t]) - sum of q_j with id_j = v),
                    dx and dw as above

A negative target or id is none; a row without any has loss and lse 0 and no
part in the gradients.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    """The cases; see the comment at each for what it stands for."""
    return [
        # the log-probability of one word while answering: latency, and the weights' way from memory
        dict(name="xent 1 row", op="xent", dtype="f16", layout="nk", T=1, V=32000, D=1024, ignored=0.0),
        # the answers of a batch of multiple-choice questions, scored: the weights are what is read
        dict(name="xent 64 rows", op="xent", dtype="bf16", layout="nk", T=64, V=131072, D=4096, ignored=0.0),
        # a fine-tuning batch of prompts and answers, sizes that divide nothing
        dict(name="xent ragged 3000 rows", op="xent", dtype="f16", layout="nk", T=3000, V=50021, D=2056, ignored=0.4),
        # a pre-training step
        dict(name="xent 8192 rows", op="xent", dtype="bf16", layout="nk", T=8192, V=131072, D=4096, ignored=0.0),
        # a small fine-tuning step, odd sizes, weights stored (D, V)
        dict(name="xent_grad 100 rows", op="xent_grad", dtype="f16", layout="kn", T=100, V=32008, D=1000, ignored=0.3, mean=True),
        # the fine-tuning batch's gradient, half of its rows being prompts
        dict(name="xent_grad ragged 5000 rows", op="xent_grad", dtype="f16", layout="nk", T=5000, V=50021, D=1544, ignored=0.5, mean=False),
        # the pre-training step's gradient
        dict(name="xent_grad 4096 rows", op="xent_grad", dtype="bf16", layout="nk", T=4096, V=131072, D=4096, ignored=0.0, mean=True),
        # a short answer beside its teacher's eight best words
        dict(name="distill 16 rows", op="distill", dtype="f16", layout="nk", T=16, V=32000, D=1024, ignored=0.0, k=8, tau=1.0),
        # a distillation step
        dict(name="distill 4096 rows", op="distill", dtype="bf16", layout="nk", T=4096, V=65536, D=2048, ignored=0.1, k=64, tau=2.0),
        # a small step, odd sizes, weights stored (D, V)
        dict(name="distill_grad 300 rows", op="distill_grad", dtype="f16", layout="kn", T=300, V=32008, D=1000, ignored=0.3, k=20, tau=1.5, mean=False),
        # the distillation step's gradient
        dict(name="distill_grad 4096 rows", op="distill_grad", dtype="bf16", layout="nk", T=4096, V=65536, D=2048, ignored=0.1, k=64, tau=2.0, mean=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges, no larger than their largest."""
    op = rng.choice(("xent", "xent_grad", "xent_grad", "distill", "distill_grad"))
    layout = rng.choice(("nk", "nk", "kn"))
    v = _log_int(rng, 8192, 131072)
    if layout == "kn" or rng.random() < 0.3:
        v = v // 8 * 8  # the rows' 16-byte pitch
    unit = rng.choice((8, 64))
    d = max(unit, _log_int(rng, 512, 4096) // unit * unit)
    most = 131072 * 4096 * (8192 if op in ("xent", "distill") else 4096)
    t = max(1, min(_log_int(rng, 1, 8192), most // (v * d)))
    case = dict(op=op, dtype=rng.choice(("f16", "bf16")), layout=layout, T=t, V=v, D=d, ignored=rng.choice((0.0, 0.1, 0.5)) if t > 16 else 0.0)
    if op.startswith("distill"):
        case.update(k=_log_int(rng, 1, 128), tau=rng.choice((1.0, 2.0, 0.5)))
    if op.endswith("_grad"):
        case["mean"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    """Rows and weights that give logits of spread 2, a few words of a row standing out by up to about 16,
    as a partly trained model's; what the gradients need from the forward pass."""
    dtype, dev = DTYPES[case["dtype"]], "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rs = np.random.RandomState(int(seed) % (2 ** 32 - 1))
    t, v, d, op = case["T"], case["V"], case["D"], case["op"]
    w = torch.randn((v, d), generator=gen, device=dev, dtype=torch.float32).mul_(2 * d ** -0.5).to(dtype)  # a row per word
    x = torch.randn((t, d), generator=gen, device=dev, dtype=torch.float32)
    # frequent words are met often: word i with odds that fall like 1 / (i + 20)
    common = lambda n: np.minimum(v - 1, (20 * ((v / 20 + 1) ** rs.random_sample(n) - 1)).astype(np.int64))  # noqa: E731
    ignored = torch.from_numpy(rs.random_sample(t) < case["ignored"]).to(dev)
    best = torch.from_numpy(common(t)).to(dev)
    lift = torch.rand((t, 1), generator=gen, device=dev) * 4
    x = (x + lift * w[best].float()).to(dtype)
    state = dict(op=op, layout=case["layout"], x=x, w=w if case["layout"] == "nk" else w.t().contiguous())
    if op.startswith("xent"):
        state["targets"] = torch.where(ignored, torch.full_like(best, -100), best).int()
        tau = 1.0
    else:
        k, tau = case["k"], case["tau"]
        ids = torch.from_numpy(common(t * k).reshape(t, k)).to(dev)
        ids[:, 0] = best
        # the teacher's logits of its best words, in falling order; now and then fewer than k of them
        logits = torch.randn((t, k), generator=gen, device=dev).mul_(2).sort(dim=1, descending=True).values + 8
        few = torch.rand((t, 1), generator=gen, device=dev) < 0.1
        place = torch.arange(k, device=dev)
        ids = torch.where((few & (place >= (k + 1) // 2)) | ignored[:, None], torch.full_like(ids, -1), ids)
        state.update(ids=ids.int().contiguous(), logits=logits.contiguous(), tau=tau)
    if op.endswith("_grad"):
        z = torch.matmul(x.float(), w.float().t()).div_(tau)
        state["lse"] = torch.where(ignored, torch.zeros((), device=dev), torch.logsumexp(z, dim=1))
        if case["mean"]:
            state["dloss"] = (1.0 / (~ignored).sum().clamp(min=1)).float().reshape(1)
        else:
            state["dloss"] = (torch.rand(t, generator=gen, device=dev) + 0.5) / t
    return state


def _teacher(ids, logits, tau):
    """(q, log q) over each row's words, 0 where there is none."""
    has = ids >= 0
    l = torch.where(has, logits.float() / tau, torch.full_like(logits, -math.inf, dtype=torch.float32))
    top = l.amax(dim=1, keepdim=True)
    l = l - torch.where(has.any(dim=1, keepdim=True), top, torch.zeros_like(top))
    q = torch.exp(l)
    total = q.sum(dim=1, keepdim=True).clamp(min=1e-30)
    return q / total, torch.where(has, l - torch.log(total), torch.zeros_like(l))


def _plain(s):
    op, x = s["op"], s["x"].float()
    w = s["w"].float() if s["layout"] == "kn" else s["w"].float().t()
    z = x @ w
    if op.startswith("xent"):
        valid = s["targets"] >= 0
        at = s["targets"].clamp(min=0).long()[:, None]
        q, log_q, tau = valid[:, None].float(), torch.zeros_like(at, dtype=torch.float32), 1.0
    else:
        valid = (s["ids"] >= 0).any(dim=1)
        at = s["ids"].clamp(min=0).long()
        tau = s["tau"]
        q, log_q = _teacher(s["ids"], s["logits"], tau)
    if not op.endswith("_grad"):
        picked = z.gather(1, at)
        z = z / tau
        top = z.amax(dim=1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
        loss = tau * tau * ((q * (log_q - picked / tau)).sum(dim=1) + lse)
        zero = torch.zeros_like(loss)
        return {"loss": torch.where(valid, loss, zero), "lse": torch.where(valid, lse, zero)}
    p = torch.exp(z / tau - s["lse"][:, None])
    p.scatter_add_(1, at, -q)
    g = p * (valid * s["dloss"] * tau)[:, None]
    dw = x.t() @ g
    return {"dx": (g @ w.t()).to(s["x"].dtype), "dw": (dw if s["layout"] == "kn" else dw.t()).to(s["x"].dtype).contiguous()}


def run(state):
    """One pass through one operator."""
    if not own:
        return _plain(state)
    import tiled_dense_gemm_gb300 as fw
    op, x, w, layout = state["op"], state["x"], state["w"], state["layout"]
    if op == "xent":
        loss, lse = fw.gemm_relu_xent(x, w, state["targets"], b_layout=layout)
        return {"loss": loss, "lse": lse}
    if op == "xent_grad":
        dx, dw = fw.gemm_relu_xent_grad(x, w, state["targets"], state["lse"], state["dloss"], b_layout=layout)
        return {"dx": dx, "dw": dw}
    if op == "distill":
        loss, lse = fw.gemm_relu_distill(x, w, state["ids"], state["logits"], temperature=state["tau"], b_layout=layout)
        return {"loss": loss, "lse": lse}
    dx, dw = fw.gemm_relu_distill_grad(x, w, state["ids"], state["logits"], state["lse"], state["dloss"],
                                       temperature=state["tau"], b_layout=layout)
    return {"dx": dx, "dw": dw}


def work(case):
    """Bytes and operations that one pass cannot do without: the rows that have a loss, the weights, the outputs.
    The logits are computed anew in the backward pass, which is given none."""
    t, v, d = case["T"], case["V"], case["D"]
    used = int(round(t * (1 - case["ignored"])))
    teacher = 8 * t * case["k"] if "k" in case else 4 * t
    read = 2 * used * d + 2 * v * d + teacher
    if not case["op"].endswith("_grad"):
        return {"bytes": read + 8 * t, "flops": 2 * used * v * d}
    return {"bytes": read + 4 * t + (4 if case["mean"] else 4 * t) + 2 * t * d + 2 * v * d, "flops": 6 * used * v * d}


def exact(case, seed):
    """The same outputs in 64 bits, by blocks of rows, each row's words one by one."""
    grad = case["op"].endswith("_grad")
    if case["T"] * case["V"] * case["D"] * (3 if grad else 1) > 8e12:
        return None
    s = prepare(case, seed)
    t, v, d = case["T"], case["V"], case["D"]
    x = s["x"].double()
    w = s["w"].double() if s["layout"] == "nk" else s["w"].double().T  # (V, D)
    if case["op"].startswith("xent"):
        ids, tau = s["targets"].long()[:, None], 1.0
        weight = torch.ones((t, 1), dtype=torch.float64, device=x.device)
    else:
        ids, tau = s["ids"].long(), case["tau"]
        raw = s["logits"].double() / tau
        raw[ids < 0] = -math.inf
        weight = torch.softmax(raw, dim=1)
    weight = torch.where(ids < 0, 0.0, weight)
    rows = torch.nonzero((ids >= 0).any(dim=1)).flatten()
    loss = torch.zeros(t, dtype=torch.float64, device=x.device)
    lse = torch.zeros_like(loss)
    dx = torch.zeros((t, d), dtype=torch.float64, device=x.device)
    dw = torch.zeros((v, d), dtype=torch.float64, device=x.device) if grad else None
    for at in rows.split(1024):
        z = torch.matmul(x[at], w.T) / tau
        if not grad:
            norm = torch.logsumexp(z, dim=1)
            lse[at] = norm
            for j in range(ids.shape[1]):
                q = weight[at, j]
                mine = norm - z.gather(1, ids[at, j].clamp(min=0)[:, None])[:, 0]
                loss[at] += tau ** 2 * (torch.xlogy(q, q) + q * mine)
            continue
        g = torch.exp(z - s["lse"].double()[at, None])
        here = torch.arange(len(at), device=x.device)
        for j in range(ids.shape[1]):
            g[here, ids[at, j].clamp(min=0)] -= weight[at, j]
        g *= (s["dloss"].double().expand(t)[at] * tau)[:, None]
        dx[at] = torch.matmul(g, w)
        dw += torch.matmul(g.T, x[at])
    if not grad:
        return {"loss": loss, "lse": lse}
    return {"dx": dx, "dw": dw if s["layout"] == "nk" else dw.T.contiguous()}
