"""Plain 64-bit forms of the serving operators (rotary positions, attention over a shared prefix, accumulated
attention weights, eviction) and the error bounds that their GPU results are held to.

Bounds.  u = 2^-24 is half a step of fp32, relative; a bf16 rounding is off by at most 2^-8, relative.
A dot product of d fp32 (or exact bf16 x bf16) terms in any order is off by at most (d + 2) u sum|q_i k_i|, which
Cauchy-Schwarz bounds by (d + 2) u |q| |k|; times 1/sqrt(d) that is the error of a logit, eps_s below, to which 4 u
of the logit's own size are added for the scaling and the exponent's argument.
"""
import math

import torch

U = 2.0 ** -24
BF = 2.0 ** -8


# ------------------------------------------------------------------ rotary positions

def rope_frequencies(R, base=10000.0, factor=1.0, orig_ctx=0, beta_fast=32.0, beta_slow=1.0):
    f = []
    for k in range(R // 2):
        w = base ** (-2.0 * k / R)
        if orig_ctx:
            g = min(1.0, max(0.0, (orig_ctx * w / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)))
            f.append(g * w + (1 - g) * w / factor)
        else:
            f.append(w / factor)
    return f


def rope_ref(x, pos, R, off, half=False, inverse=False, out_scale=1.0, **kw):
    """x [B][T][H][d] (any dtype), pos [B][T] ints: the rotated rows in float64."""
    y = x.double().clone()
    f = rope_frequencies(R, **kw)
    ang = torch.tensor([[[math.fmod(p * w, 2 * math.pi) for w in f] for p in row] for row in pos.tolist()],
                       dtype=torch.float64)
    c, s = ang.cos()[:, :, None] * out_scale, ang.sin()[:, :, None] * (-out_scale if inverse else out_scale)
    i0 = torch.arange(off, off + R // 2) if half else torch.arange(off, off + R, 2)
    i1 = i0 + (R // 2 if half else 1)
    a, b = x[..., i0].double(), x[..., i1].double()
    y[..., i0] = a * c - b * s
    y[..., i1] = b * c + a * s
    return y


def rope_bound(x, ref, pos, R, off, out_scale=1.0, rounding=U):
    """Elementwise: each of the two products carries the error of its cosine (the angle in turns is rounded to fp32
    once, 2^-24 of up to half a turn, plus 2 ulp of sincospi and one of the scale), two fp32 roundings, and the
    output's own.  The reference's own angle, a double product of up to 2^40 rad, adds pos 2^-52."""
    big = x.double().abs().amax(-1, keepdim=True) * out_scale
    err = big * 2 * (math.pi * U + 6 * U) + big * 2 * pos.double().abs()[:, :, None, None] * 2.0 ** -52
    return err + ref.abs() * rounding


# ------------------------------------------------------------------ shared-prefix attention, weights

def query_positions(lens, n_q):
    return [[n - n_q + j for j in range(n_q)] for n in lens]


def candidates(b, t, *, prefix, own, ring, counts, entries, m, W):
    """The rows (float64) that a query of sequence b at position t attends to, and which own slots are among them."""
    Np = prefix.shape[0]
    if t < 0 or (t + 1) // m < Np:
        return torch.zeros((0, own.shape[-1]), dtype=torch.float64), []
    ent = entries[b] if entries is not None else [Np + i for i in range(own.shape[1])]
    slots = [i for i in range(counts[b]) if 0 <= ent[i] and m * (ent[i] + 1) <= t + 1]
    win = [p % ring.shape[1] for p in range(max(0, t - W + 1), t + 1)] if W else []
    return torch.cat((prefix, own[b, slots], ring[b, win])).double(), slots


def shared_ref(q, prefix, own, ring, *, lens, counts, entries, m, W, sink=None, rope_dims=0, rope_base=10000.0,
               p_rounding=U, out_rounding=U):
    """out and lse in float64, and elementwise bounds for both."""
    B, T, H, d = q.shape
    out, lse = torch.zeros((B, T, H, d), dtype=torch.float64), torch.full((B, T, H), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        for j, t in enumerate(query_positions(lens, T)[b]):
            kv, _ = candidates(b, t, prefix=prefix, own=own, ring=ring, counts=counts, entries=entries, m=m, W=W)
            if len(kv) == 0:
                continue
            qq = q[b, j].double()
            s = qq @ kv.T / math.sqrt(d)
            eps = (d + 2) * U * qq.norm(dim=1, keepdim=True) * kv.norm(dim=1) / math.sqrt(d) + 4 * U * s.abs()
            logits = s if sink is None else torch.cat((s, sink.double()[:, None]), 1)
            z = torch.logsumexp(logits, 1)
            p = (s - z[:, None]).exp()
            o = p @ kv
            e = eps.amax(1)
            n = len(kv) + 8
            lse[b, j] = z
            # the log of a sum of n terms, each off by e^(+-e), summed in fp32, the log's and the maximum's rounding
            tol_l[b, j] = 1.01 * e + n * U + 4 * U * z.abs() + 4 * U
            # numerator: every p off by (e^(2 e) - 1) + its rounding + n u of the sum; then the division and rounding
            rel = 2.02 * e + n * 2 * U + p_rounding
            to = (p @ kv.abs()) * rel[:, None]
            if rope_dims:
                R, r0 = rope_dims, d - rope_dims
                ang = torch.tensor([math.fmod(-t * rope_base ** (-2.0 * k / R), 2 * math.pi) for k in range(R // 2)],
                                   dtype=torch.float64)
                x, y = o[:, r0::2].clone(), o[:, r0 + 1::2].clone()
                o[:, r0::2], o[:, r0 + 1::2] = x * ang.cos() - y * ang.sin(), y * ang.cos() + x * ang.sin()
                both = to[:, r0::2] + to[:, r0 + 1::2] + 8 * U * (x.abs() + y.abs())
                both = both + (x.abs() + y.abs()) * abs(t) * 2.0 ** -50
                to[:, r0::2], to[:, r0 + 1::2] = both, both
            out[b, j] = o
            tol_o[b, j] = to + o.abs() * out_rounding + 1e-30
    return out, lse, tol_o, tol_l


def weights_ref(q, own, lse, weights, *, n_prefix, lens, counts, entries, m, decay):
    """The new weights of the held slots in float64 (others: nan), and their bounds."""
    B, T, H, d = q.shape
    rows = own.shape[1]
    got = torch.full((B, rows), math.nan, dtype=torch.float64)
    tol = torch.zeros_like(got)
    for b in range(B):
        n = counts[b]
        got[b, :n] = weights[b, :n].double() * decay if decay else 0.0
        tol[b, :n] = got[b, :n].abs() * 2 * U
        for j, t in enumerate(query_positions(lens, T)[b]):
            if t < 0 or (t + 1) // m < n_prefix:
                continue
            ent = entries[b] if entries is not None else [n_prefix + i for i in range(rows)]
            for i in range(n):
                if ent[i] < 0 or m * (ent[i] + 1) > t + 1:
                    continue
                k = own[b, i].double()
                s = q[b, j].double() @ k / math.sqrt(d)
                z = lse[b, j].double()
                live = z != -math.inf
                p = torch.where(live, (s - z).exp(), 0.0)
                eps = (d + 2) * U * q[b, j].double().norm(dim=1) * k.norm() / math.sqrt(d) + 4 * U * (s.abs() + z.abs().clamp(max=1e9))
                got[b, i] += p.sum()
                tol[b, i] += (p * (1.02 * torch.where(live, eps, 0.0) + (T * H + 8) * U)).sum()
    return got, tol


# ------------------------------------------------------------------ eviction

def evict_ref(weights, counts, budget, first, recent):
    """The kept slots of every sequence."""
    kept = []
    for b, n in enumerate(counts):
        fixed = {i for i in range(n) if i < first or i >= n - recent}
        if n <= budget:
            kept.append(list(range(n)))
            continue
        w = weights[b].tolist()
        rest = sorted((i for i in range(n) if i not in fixed), key=lambda i: (math.isnan(w[i]), -w[i] if not math.isnan(w[i]) else 0.0, i))
        kept.append(sorted(list(fixed) + rest[: budget - len(fixed)]))
    return kept
