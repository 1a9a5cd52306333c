"""The measured cases of the loss operators on an output head's product.

A language model ends in the product Z = X·Wᵀ of its last hidden states X
(T×D, a row a token) with the head's weight W (V×D, a row a word of the
vocabulary), and a loss on the rows of Z.  Z is the largest matrix of a
training step; the operators measured here take X and W and never hold Z.

* cross entropy: loss_t = lse_t - z_{t,y_t}, lse_t = log sum_v exp z_tv;
* distillation from a teacher's top logits: with a temperature s, q_t the
  softmax of the teacher's K logits over s and z the student's logits over s,
  loss_t = s²·sum_k q_tk·(log q_tk - (z_{t,id_tk} - lse_t)).

A "forward" case gives the losses of the rows, as evaluation and scoring use
them; a "step" case is what a training program does with the operator: the
mean loss and the gradients of X and W.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100


def listed():
    return [
        # cross entropy
        # the log-probability of one chosen token while serving: latency, W read once
        dict(name="score one token", op="ce", step=False, T=1, V=32000, D=4096, type="bf16"),
        # a few candidate tokens of a small model scored together, odd sizes
        dict(name="score 21 tokens odd", op="ce", step=False, T=21, V=10007, D=520, type="fp16"),
        # the loss of a held-out batch
        dict(name="evaluate", op="ce", step=False, T=4096, V=32000, D=4096, type="bf16"),
        # a training step of a small model on a ragged float32 product (3000x1000 times 1000x5000)
        dict(name="train ragged fp32", op="ce", step=True, T=3000, V=5000, D=1000, type="fp32"),
        # fine-tuning on one short sequence
        dict(name="train few rows fp16", op="ce", step=True, T=33, V=8192, D=512, type="fp16"),
        # an ordinary training step
        dict(name="train", op="ce", step=True, T=4096, V=32768, D=2048, type="bf16"),
        # a large vocabulary and a wide model
        dict(name="train largest", op="ce", step=True, T=8192, V=131072, D=4096, type="bf16"),
        # distillation
        # how far a student is from its teacher on a few tokens
        dict(name="compare 16 tokens", op="kd", step=False, T=16, V=32000, D=1024, K=16, temperature=1.0, type="bf16"),
        # the distillation loss of a held-out batch
        dict(name="distill evaluate", op="kd", step=False, T=2048, V=50001, D=1024, K=100, temperature=2.0, type="fp16"),
        # a distillation step in float32 on a small student
        dict(name="distill fp32", op="kd", step=True, T=512, V=16384, D=1024, K=20, temperature=1.0, type="fp32"),
        # a distillation step, sizes that no tile divides
        dict(name="distill odd", op="kd", step=True, T=777, V=20011, D=1000, K=33, temperature=3.0, type="bf16"),
        # an ordinary distillation step
        dict(name="distill", op="kd", step=True, T=4096, V=32768, D=2048, K=64, temperature=2.0, type="bf16"),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["ce", "kd"]), step=rng.random() < 0.6, T=_between(rng, 1, 8192), V=_between(rng, 1000, 131072),
                 D=_between(rng, 64, 4096), type=rng.choice(["bf16", "fp16", "fp32"]))
        if rng.random() < 0.6:  # models mostly have widths that are multiples of 64
            c["D"] = max(64, c["D"] // 64 * 64)
        if c["op"] == "kd":
            c["K"] = _between(rng, 1, 128)
            c["temperature"] = rng.choice([1.0, 1.5, 2.0, 4.0])
        if c["T"] * c["V"] * c["D"] * (8 if c["type"] == "fp32" else 1) <= 8192 * 131072 * 4096:
            return c


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, V, D, kind = case["T"], case["V"], case["D"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)

    s = dict(case=case)
    s["X"] = normal(T, D).to(kind)
    s["W"] = (normal(V, D) * (2.0 / math.sqrt(D))).to(kind)  # logits of about N(0, 4)
    if case["op"] == "ce":
        target = torch.randint(0, V, (T,), generator=g, device="cuda")
        if T >= 16:  # padding and prompt tokens that do not count
            target[uniform(T) < 0.08] = IGNORE
        s["target"] = target
    else:
        K = case["K"]
        # one word of each K-th part of the vocabulary, in an order of its own for each row
        at = (torch.arange(K, device="cuda") + uniform(T, K).double() * 0.999) * (V / K)
        order = uniform(T, K).argsort(dim=1)
        s["ids"] = at.long().clamp_(max=V - 1).gather(1, order)
        top = (normal(T, K) * 2.0 + 6.0).sort(dim=1, descending=True).values
        if T >= 16:  # rows with fewer entries, and rows with none
            left = torch.where(uniform(T) < 0.1, uniform(T) * K, torch.full((T,), float(K), device="cuda"))
            top[torch.arange(K, device="cuda") >= left[:, None].floor()] = float("-inf")
        s["top"] = top.to(kind)
    if case["step"]:
        s["X"].requires_grad_()
        s["W"].requires_grad_()
    return s


def _soft(top, scale):
    """The teacher's probabilities over its kept entries, their logarithms (0 where there is none), and which rows have any."""
    kept = top > float("-inf")
    some = kept.any(dim=1)
    t = torch.where(kept, top * scale, 0.0)
    high = torch.where(kept, t, float("-inf")).amax(dim=1, keepdim=True)
    t = torch.where(kept, t - torch.where(some[:, None], high, 0.0), 0.0)
    e = torch.where(kept, torch.exp(t), 0.0)
    total = torch.where(some, e.sum(dim=1), 1.0)[:, None]
    return e / total, torch.where(kept, t - torch.log(total), 0.0), kept, some


def _plain(s):
    case, kind = s["case"], s["X"].dtype
    x, w = s["X"].detach().float(), s["W"].detach().float()
    scale = 1.0 / case.get("temperature", 1.0)
    z = x @ w.t()
    if scale != 1.0:
        z = z * scale
    high = z.amax(dim=1, keepdim=True)
    lse = torch.log(torch.exp(z - high).sum(dim=1)) + high[:, 0]
    if case["op"] == "ce":
        some = s["target"] != IGNORE
        at = torch.where(some, s["target"], 0)[:, None]
        loss = torch.where(some, lse - z.gather(1, at)[:, 0], 0.0)
        q = some.float()[:, None]
    else:
        at = s["ids"]
        q, log_q, kept, some = _soft(s["top"].float(), scale)
        picked = torch.where(kept, z.gather(1, at), 0.0)
        loss = (q * (log_q - (picked - lse[:, None]))).sum(dim=1) / scale ** 2
        loss = torch.where(some, loss, 0.0)
    if not case["step"]:
        return (loss, lse) if case["op"] == "ce" else (loss, lse, picked)
    count = some.sum().clamp(min=1)
    p = torch.exp(z - lse[:, None])
    p[~some] = 0.0
    p.scatter_add_(1, at, -q)
    p *= 1.0 / (scale * count)
    return loss.sum() / count, (p @ w).to(kind), (p.t() @ x).to(kind)


def _own(s):
    import tiled_gemm_tgemm_amd as tg

    case = s["case"]
    if case["op"] == "ce":
        if not case["step"]:
            return tg.linear_cross_entropy_forward(s["X"], s["W"], s["target"], ignore_index=IGNORE)
        loss = tg.linear_cross_entropy(s["X"], s["W"], s["target"], ignore_index=IGNORE)
    else:
        if not case["step"]:
            return tg.linear_distillation_forward(s["X"], s["W"], s["ids"], s["top"], temperature=case["temperature"])
        loss = tg.linear_distillation(s["X"], s["W"], s["ids"], s["top"], temperature=case["temperature"])
    dX, dW = torch.autograd.grad(loss, (s["X"], s["W"]))
    return loss.detach(), dX, dW


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    T, V, D = case["T"], case["V"], case["D"]
    size = 4 if case["type"] == "fp32" else 2
    read = (T + V) * D * size + (T * 8 if case["op"] == "ce" else T * case["K"] * (8 + size))
    if case["step"]:  # the logits' product and one for each gradient; the gradients are as large as X and W
        return {"bytes": read + (T + V) * D * size + 4, "flops": 6 * T * V * D}
    return {"bytes": read + T * 8 + (T * case["K"] * 4 if case["op"] == "kd" else 0), "flops": 2 * T * V * D}


def exact(case, seed):
    s = prepare(case, seed)
    T, V, step = case["T"], case["V"], case["step"]
    tau = float(case.get("temperature", 1.0))
    X, W = s["X"].detach().double(), s["W"].detach().double()
    if case["op"] == "ce":
        counts = s["target"] >= 0
    else:
        counts = ~torch.isinf(s["top"]).all(dim=1)
    n = max(1, int(counts.sum()))
    losses, sums, picks = [], [], []
    dX, dW = (torch.empty_like(X), torch.zeros_like(W)) if step else (None, None)
    rows = max(1, min(T, (1 << 27) // V))
    for lo in range(0, T, rows):
        x, c = X[lo:lo + rows], counts[lo:lo + rows]
        z = torch.matmul(x, W.t()) / tau
        lse = torch.logsumexp(z, dim=1)
        wanted = torch.zeros_like(z)  # the distribution that the row is held to
        if case["op"] == "ce":
            y = s["target"][lo:lo + rows]
            r = torch.arange(len(y), device=y.device)[c]
            wanted[r, y[c]] = 1.0
            losses.append(torch.where(c, lse - (wanted * z).sum(dim=1), 0.0))
        else:
            ids, top = s["ids"][lo:lo + rows], s["top"][lo:lo + rows].double() / tau
            q = torch.where(c[:, None], torch.softmax(top, dim=1), 0.0)
            wanted.scatter_add_(1, ids, q)
            log_p = z.gather(1, ids) - lse[:, None]
            losses.append(tau * tau * (torch.xlogy(q, q) - q * log_p).sum(dim=1))
            picks.append(torch.where(torch.isinf(top), 0.0, z.gather(1, ids)))
        sums.append(lse)
        if step:
            d = torch.softmax(z, dim=1)
            d -= wanted
            d *= (c.double() * tau / n)[:, None]
            dX[lo:lo + rows] = torch.matmul(d, W)
            dW += torch.matmul(d.t(), x)
            del d
        del z, wanted
    loss, lse = torch.cat(losses), torch.cat(sums)
    if step:
        return loss.sum() / n, dX, dW
    return (loss, lse) if case["op"] == "ce" else (loss, lse, torch.cat(picks))
