"""Plain 64-bit forms of the loss operators, on torch tensors of any device.

Every function takes the operators' own inputs (BF16 / FP32 / integers) and
returns losses, gradients and the magnitudes that the tests' tolerances are
made of.
"""
import math

import torch


def linear_cross_entropy(h, W, target, g):
    """loss [T], dh, dW, the summed magnitudes |d| |W| and |d|^T |h|, and max over v of sum_i |h_ti W_vi|."""
    h, W = h.double(), W.double()
    T, V = h.shape[0], W.shape[0]
    has = (target >= 0) & (target < V)
    at = torch.where(has, target, 0).long()[:, None]
    z = h @ W.t()
    lse = torch.logsumexp(z, 1)
    loss = torch.where(has, lse - z.gather(1, at)[:, 0], 0.0)
    d = torch.exp(z - lse[:, None])
    d.scatter_add_(1, at, -torch.ones(T, 1, dtype=torch.float64, device=h.device))
    # the target's p - 1 without cancellation
    rest = torch.where(torch.arange(V, device=h.device)[None] == at, 0.0, d).sum(1, keepdim=True)
    d.scatter_(1, at, -rest)
    d *= (has.double() * g)[:, None]
    mag = h.abs() @ W.abs().t()
    return loss, d @ W, d.t() @ h, d.abs() @ W.abs(), d.abs().t() @ h.abs(), mag.amax(1)


def distill(logits, target, t_val, t_idx, tau, w_ce, w_kd):
    """ce [R], kd [R], dz, the magnitude of dz's terms and of kd's."""
    z = logits.double()
    R, V = z.shape
    dz, mag = torch.zeros_like(z), torch.zeros_like(z)
    ce, kd, kmag = (torch.zeros(R, dtype=torch.float64, device=z.device) for _ in range(3))
    for r in range(R):
        if target is not None and 0 <= int(target[r]) < V:
            t = int(target[r])
            lp = torch.log_softmax(z[r], 0)
            ce[r] = -lp[t]
            p = lp.exp()
            mag[r] += abs(w_ce) * p
            dz[r] += w_ce * p
            dz[r, t] -= w_ce * p[t] + w_ce * (p.sum() - p[t])
        ids = t_idx[r].long()
        keep = (ids >= 0) & (ids < V) & (t_val[r] != -math.inf)
        if bool(keep.any()):
            ids, lq = ids[keep], torch.log_softmax(t_val[r][keep].double() / tau, 0)
            q = lq.exp()
            lp = torch.log_softmax(z[r] / tau, 0)
            terms = torch.where(q > 0, q * (lq - lp[ids]), 0.0)
            kd[r], kmag[r] = terms.sum(), (q * (lq.abs() + 1)).sum() + terms.abs().sum()
            dz[r] += w_kd / tau * lp.exp()
            dz[r].index_add_(0, ids, -w_kd / tau * q)
            mag[r] += abs(w_kd) / tau * lp.exp()
            mag[r].index_add_(0, ids, abs(w_kd) / tau * q)
    return ce, kd, dz, mag, kmag


def router_balance(logits, idx, valid, S, alpha, z_coef):
    """loss [2], counts, prob, dlogits and the magnitude of its terms."""
    z = logits.double()
    T, E = z.shape
    G, k = T // S, idx.shape[1]
    loss = torch.zeros(2, dtype=torch.float64, device=z.device)
    counts = torch.zeros(G, E, dtype=torch.int32, device=z.device)
    prob = torch.zeros(G, E, dtype=torch.float64, device=z.device)
    d, mag = torch.zeros_like(z), torch.zeros_like(z)
    for g in range(G):
        rows = torch.arange(g * S, (g + 1) * S, device=z.device)
        if valid is not None:
            rows = rows[valid[rows] != 0]
        n = rows.numel()
        if n == 0:
            continue
        c = idx[rows].long().reshape(-1)
        c = c[(c >= 0) & (c < E)]
        counts[g] = torch.bincount(c, minlength=E)
        f = counts[g].double() / (n * k)
        p, lse = torch.softmax(z[rows], 1), torch.logsumexp(z[rows], 1)
        prob[g] = p.mean(0)
        loss[0] += alpha * E / G * (f * prob[g]).sum()
        loss[1] += z_coef / G * (lse * lse).mean()
        cb, cz = alpha * E / (G * n), 2 * z_coef / (G * n)
        mean = (p * f).sum(1, keepdim=True)
        d[rows] = cb * p * (f - mean) + cz * lse[:, None] * p
        mag[rows] = abs(cb) * p * (f + mean) + abs(cz) * (lse.abs() + z[rows].abs().amax(1))[:, None] * p
    return loss, counts, prob, d, mag
