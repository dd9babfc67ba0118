"""Cases and plain forms of the loss operators: linear cross entropy, distillation from a teacher's top logits, and the
router's balance loss.

``listed()`` and ``draw(rng)`` give cases, ``prepare`` makes a case's inputs and the buffers a training program keeps, ``run``
makes one pass (elementary torch operations in 32 bits, or the library's calls where ``own`` is true), ``work`` counts what a
pass cannot do without and ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the head of the tiny decoder: launches and latency
        dict(name="lce tiny", op="lce", T=256, H=256, V=1024, grads=True),
        # the head of the 1.2B decoder, its whole step of 4 x 2048 tokens
        dict(name="lce 1.2b", op="lce", T=8192, H=2048, V=32000, grads=True),
        # the head of the 7.6B decoder, one micro-batch of 4096 tokens
        dict(name="lce 7.6b", op="lce", T=4096, H=3584, V=152064, grads=True),
        # a few scored tokens against the same head: the weights are read and written for almost no work
        dict(name="lce few", op="lce", T=5, H=3584, V=152064, grads=True),
        # evaluation (no gradients) of a ragged batch with the MoE decoder's head
        dict(name="lce eval", op="lce", T=1777, H=2880, V=201088, grads=False),
        # a small student and a short list
        dict(name="kd tiny", op="kd", rows=256, V=1024, K=8, tau=1.0, hard=True),
        # the 1.2B decoder's step, teacher and targets mixed at a temperature
        dict(name="kd 1.2b", op="kd", rows=8192, V=32000, K=32, tau=2.0, hard=True),
        # a vocabulary of odd size, teacher alone
        dict(name="kd odd", op="kd", rows=1001, V=50257, K=50, tau=1.5, hard=False),
        # one micro-batch of the 7.6B decoder, a long list
        dict(name="kd 7.6b", op="kd", rows=4096, V=152064, K=128, tau=1.0, hard=True),
        # the tiny MoE decoder, a loss for each of its two sequences
        dict(name="bal tiny", op="bal", T=256, S=128, E=8, k=2, masked=False),
        # the MoE decoder's step of 4 sequences of 4096 tokens, padded at their ends
        dict(name="bal moe", op="bal", T=16384, S=4096, E=32, k=4, masked=True),
        # many small experts over one long sequence
        dict(name="bal 128", op="bal", T=131072, S=131072, E=128, k=8, masked=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("lce", "kd", "bal"))
    if op == "lce":
        H = 8 * _log_int(rng, 8, 448)
        return dict(op=op, T=_log_int(rng, 1, 4096), H=H, V=_log_int(rng, 256, 152064), grads=rng.random() < 0.75)
    if op == "kd":
        V = _log_int(rng, 256, 152064)
        return dict(op=op, rows=_log_int(rng, 1, 4096), V=V, K=_log_int(rng, 1, 128),
                    tau=rng.choice((1.0, 2.0, round(rng.uniform(0.5, 4.0), 3))), hard=rng.random() < 0.5)
    S = _log_int(rng, 1, 8192)
    E = _log_int(rng, 2, 128)
    return dict(op=op, T=S * rng.randint(1, 16), S=S, E=E, k=rng.randint(1, min(8, E)), masked=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=g, **dev)

    s = dict(case)
    if case["op"] == "lce":
        T, H, V = case["T"], case["H"], case["V"]
        # normalised activations; weights that give logits of a standard deviation of about 2.5
        s["h"] = normal(T, H).to(BF16)
        s["W"] = (normal(V, H) * (2.5 / math.sqrt(H))).to(BF16)
        target = torch.randint(0, V, (T,), generator=g, dtype=torch.int32, **dev)
        target[15::16] = -1  # rows without a target: a sequence's last token, padding
        s["target"] = target
        s["inv_norm"] = 1.0 / max(1, T - T // 16)
        s["row_loss"] = torch.empty(T, **dev)
        s["dh"] = torch.empty_like(s["h"]) if case["grads"] else None
        s["dW"] = torch.empty_like(s["W"]) if case["grads"] else None
    elif case["op"] == "kd":
        R, V, K = case["rows"], case["V"], case["K"]
        z = normal(R, V) * 2.5
        s["logits"] = z.to(BF16)
        # the teacher agrees with the student in part: its K largest logits, sorted
        top = torch.topk(z.add_(normal(R, V)), K, dim=1)
        del z
        s["t_val"], ids = top.values.contiguous(), top.indices.to(torch.int32)
        if K > 2:
            ids[3::8, K - K // 3:] = -1  # shorter lists
        ids[7::32] = -1  # rows that the teacher left out
        s["t_idx"] = ids.contiguous()
        s["target"] = None
        if case["hard"]:
            target = torch.randint(0, V, (R,), generator=g, dtype=torch.int32, **dev)
            target[::3] = s["t_idx"][::3, 0]  # often the teacher's first choice
            target[15::16] = -1
            s["target"] = target
        s["w_ce"] = 0.5 / R if case["hard"] else 0.0
        s["w_kd"] = 0.5 * case["tau"] ** 2 / R
        s["row_ce"] = torch.empty(R, **dev) if case["hard"] else None
        s["row_kd"] = torch.empty(R, **dev)
        s["dlogits"] = torch.empty_like(s["logits"])
    else:
        T, S, E, k = case["T"], case["S"], case["E"], case["k"]
        s["logits"] = normal(T, E) * 1.5 + normal(E)  # some experts are liked more than others
        s["idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        s["valid"] = None
        if case["masked"]:  # each sequence is padded at its end, a different length each
            length = torch.randint(0, S + 1, (T // S, 1), generator=g, **dev)
            s["valid"] = (torch.arange(S, **dev)[None, :] < length).to(torch.uint8).reshape(T).contiguous()
        s["alpha"], s["z_coef"] = 0.01, 0.001
        s["loss"] = torch.empty(2, **dev)
        s["counts"] = torch.empty(T // S, E, dtype=torch.int32, **dev)
        s["prob"] = torch.empty(T // S, E, **dev)
        s["dlogits"] = torch.empty(T, E, dtype=BF16, **dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"lce": _plain_lce, "kd": _plain_kd, "bal": _plain_bal}[s["op"]](s)


def _scratch(s, nbytes):
    """The workspace a program keeps beside its buffers."""
    if "scratch" not in s:
        s["scratch"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s["scratch"]


def _run_own(s):
    from host_memory_centric_gb300 import ops

    if s["op"] == "lce":
        T, H = s["h"].shape
        V = s["W"].shape[0]
        scratch = _scratch(s, ops.linear_cross_entropy_scratch_bytes(T, H, V, s["grads"]))
        ops.linear_cross_entropy(s["h"], s["W"], s["target"], s["inv_norm"], s["row_loss"], s["dh"], s["dW"], scratch)
        return [s["row_loss"], s["dh"], s["dW"]] if s["grads"] else [s["row_loss"]]
    if s["op"] == "kd":
        ops.distill_topk(s["logits"], s["target"], s["t_val"], s["t_idx"], s["tau"], s["w_ce"], s["w_kd"], s["row_ce"],
                         s["row_kd"], s["dlogits"])
        return [s["row_kd"], s["dlogits"]] + ([s["row_ce"]] if s["hard"] else [])
    T, E = s["logits"].shape
    scratch = _scratch(s, ops.router_balance_scratch_bytes(T, s["S"], E))
    ops.router_balance(s["logits"], s["idx"], s["valid"], s["S"], s["alpha"], s["z_coef"], s["loss"], s["counts"],
                       s["prob"], s["dlogits"], scratch)
    return [s["loss"], s["counts"], s["prob"], s["dlogits"]]


def _plain_lce(s):
    h, W = s["h"].float(), s["W"].float()
    has = s["target"] >= 0
    at = s["target"].long().clamp(min=0)[:, None]
    z = h @ W.t()
    m = z.amax(dim=1, keepdim=True)
    e = (z - m).exp()
    total = e.sum(dim=1, keepdim=True)
    loss = (m + total.log() - z.gather(1, at))[:, 0]
    loss = torch.where(has, loss, torch.zeros_like(loss))
    if not s["grads"]:
        return [loss]
    d = e.div_(total)
    d.scatter_add_(1, at, torch.full_like(total, -1.0))
    d.mul_(has[:, None] * s["inv_norm"])
    return [loss, (d @ W).to(BF16), (d.t() @ h).to(BF16)]


def _plain_kd(s):
    z, tau = s["logits"].float(), s["tau"]
    ids = s["t_idx"].long()
    filled = ids >= 0
    some = filled.any(dim=1, keepdim=True)
    at = ids.clamp(min=0)
    # the teacher's distribution over the slots that are filled
    y = torch.where(filled, s["t_val"] / tau, torch.full_like(s["t_val"], -math.inf))
    top = torch.where(some, y.amax(dim=1, keepdim=True), torch.zeros_like(y[:, :1]))
    q = (y - top).exp()
    norm = torch.where(some, q.sum(dim=1, keepdim=True), torch.ones_like(y[:, :1]))
    q = q / norm
    log_q = torch.where(filled, y - top - norm.log(), torch.zeros_like(y))
    m = z.amax(dim=1, keepdim=True)
    e = ((z - m) / tau).exp()
    total = e.sum(dim=1, keepdim=True)
    log_p = (z.gather(1, at) - m) / tau - total.log()
    kd = torch.where(filled, q * (log_q - log_p), torch.zeros_like(q)).sum(dim=1)
    d = e.div_(total)
    d.scatter_add_(1, at, -q)
    d.mul_(some * (s["w_kd"] / tau))
    if not s["hard"]:
        return [kd, d.to(BF16)]
    has = s["target"] >= 0
    tat = s["target"].long().clamp(min=0)[:, None]
    e = (z - m).exp()
    total = e.sum(dim=1, keepdim=True)
    ce = (m + total.log() - z.gather(1, tat))[:, 0]
    ce = torch.where(has, ce, torch.zeros_like(ce))
    e.div_(total)
    e.scatter_add_(1, tat, torch.full_like(total, -1.0))
    d.add_(e.mul_(has[:, None] * s["w_ce"]))
    return [kd, d.to(BF16), ce]


def _plain_bal(s):
    z = s["logits"]
    T, E = z.shape
    S, k = s["S"], s["k"]
    G = T // S
    use = torch.ones(T, 1, device=z.device) if s["valid"] is None else s["valid"].float()[:, None]
    n = use.reshape(G, S).sum(dim=1)[:, None].clamp(min=1.0)
    hot = (s["idx"].reshape(T * k, 1) == torch.arange(E, device=z.device, dtype=torch.int32)).reshape(T, k, E)
    counts = (hot.sum(dim=1) * use.to(torch.int64)).reshape(G, S, E).sum(dim=1)
    f = counts.float() / (n * k)
    m = z.amax(dim=1, keepdim=True)
    e = (z - m).exp()
    total = e.sum(dim=1, keepdim=True)
    lse = m + total.log()
    p = e / total
    prob = (p * use).reshape(G, S, E).sum(dim=1) / n
    balance = s["alpha"] * E / G * (f * prob).sum()
    zloss = s["z_coef"] / G * ((lse * lse * use).reshape(G, S).sum(dim=1, keepdim=True) / n).sum()
    ft = f.repeat_interleave(S, dim=0)
    nt = n.repeat_interleave(S, dim=0)
    mean = (ft * p).sum(dim=1, keepdim=True)
    d = (s["alpha"] * E / G * p * (ft - mean) + 2.0 * s["z_coef"] / G * lse * p) * use / nt
    return [torch.stack([balance, zloss]), counts.to(torch.int32), prob, d.to(BF16)]


# ------------------------------------------------------------------ work and 64-bit values
def work(case):
    if case["op"] == "lce":
        T, H, V = case["T"], case["H"], case["V"]
        both = 2 if case["grads"] else 1
        return {"bytes": 2 * (T + V) * H * both + 8 * T, "flops": 2 * T * H * V * (3 if case["grads"] else 1)}
    if case["op"] == "kd":
        R, V, K = case["rows"], case["V"], case["K"]
        return {"bytes": 4 * R * V + 8 * R * K + (12 if case["hard"] else 4) * R, "flops": R * V * (12 if case["hard"] else 7)}
    T, S, E, k = case["T"], case["S"], case["E"], case["k"]
    return {"bytes": 6 * T * E + 4 * T * k + (T if case["masked"] else 0) + 8 * (T // S) * E + 8, "flops": 12 * T * E}


def exact(case, seed):
    s = prepare(case, seed)
    return {"lce": _exact_lce, "kd": _exact_kd, "bal": _exact_bal}[case["op"]](s)


def _exact_lce(s):
    # the 64-bit products of the largest case take about 15 seconds
    W = s["W"].double()
    T, grads = s["h"].shape[0], s["grads"]
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    dh = torch.zeros(s["h"].shape, dtype=torch.float64, device="cuda") if grads else None
    dW = torch.zeros_like(W) if grads else None
    for a in range(0, T, 1024):
        h, target = s["h"][a:a + 1024].double(), s["target"][a:a + 1024].long()
        rows = torch.nonzero(target >= 0)[:, 0]
        if rows.numel() == 0:
            continue
        log_p = torch.log_softmax(torch.mm(h[rows], W.t()), dim=1)
        loss[a + rows] = -log_p[torch.arange(rows.numel(), device="cuda"), target[rows]]
        if grads:
            d = log_p.exp_()
            d[torch.arange(rows.numel(), device="cuda"), target[rows]] -= 1.0
            d *= s["inv_norm"]
            dh[a + rows] = torch.mm(d, W)
            dW.addmm_(d.t(), h[rows])
    return [loss, dh, dW] if grads else [loss]


def _exact_kd(s):
    R, V = s["logits"].shape
    tau = s["tau"]
    kd = torch.zeros(R, dtype=torch.float64, device="cuda")
    ce = torch.zeros(R, dtype=torch.float64, device="cuda")
    grad = torch.zeros(R, V, dtype=torch.float64, device="cuda")
    for a in range(0, R, 1024):
        z, ids = s["logits"][a:a + 1024].double(), s["t_idx"][a:a + 1024].long()
        y = s["t_val"][a:a + 1024].double() / tau
        y[ids < 0] = -math.inf
        taught = torch.nonzero((ids >= 0).any(dim=1))[:, 0]
        at, y = ids[taught].clamp(min=0), y[taught]
        log_q = torch.log_softmax(y, dim=1)
        q = log_q.exp()
        log_p = torch.log_softmax(z[taught] / tau, dim=1)
        terms = q * (log_q - log_p.gather(1, at))
        terms[q == 0] = 0.0
        kd[a + taught] = terms.sum(dim=1)
        grad[a + taught] += s["w_kd"] / tau * log_p.exp().scatter_add(1, at, -q)
        if s["hard"]:
            target = s["target"][a:a + 1024].long()
            rows = torch.nonzero(target >= 0)[:, 0]
            log_p = torch.log_softmax(z[rows], dim=1)
            ce[a + rows] = -log_p.gather(1, target[rows, None])[:, 0]
            log_p.exp_().scatter_add_(1, target[rows, None], torch.full_like(log_p[:, :1], -1.0))
            grad[a + rows] += s["w_ce"] * log_p
    return [kd, grad] + ([ce] if s["hard"] else [])


def _exact_bal(s):
    z = s["logits"].double()
    T, E = z.shape
    S, k = s["S"], s["k"]
    G = T // S
    use = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"] != 0
    group = torch.arange(T, device="cuda") // S
    n = torch.bincount(group[use], minlength=G).double()
    slots = (group[use, None] * E + s["idx"][use].long()).reshape(-1)
    counts = torch.bincount(slots, minlength=G * E).reshape(G, E)
    some = n > 0
    share = 1.0 / torch.where(some, n, torch.ones_like(n))  # one valid token's weight in its group
    f = counts * share[:, None] / k
    lse = torch.logsumexp(z, dim=1)
    p = torch.softmax(z, dim=1)
    w = share[group] * use
    prob = torch.zeros(G, E, dtype=torch.float64, device="cuda").index_add_(0, group, p * w[:, None])
    loss = torch.stack([s["alpha"] * E / G * (f * prob).sum(), s["z_coef"] / G * (lse.square() * w).sum()])
    dp = s["alpha"] * E / G * f[group]
    d = p * (dp - (dp * p).sum(dim=1, keepdim=True)) + 2 * s["z_coef"] / G * lse[:, None] * p
    return [loss, counts, prob, d * w[:, None]]
