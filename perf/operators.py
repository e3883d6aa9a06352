"""Cases, inputs and plain forms of the serving operators around the compressed-attention path.

Four operators that a program serving a batch of long sequences runs next to compression, indexing and attention:

  rope      rotary positions of queries, K=V rows and indexer queries, several streams in one call, and its gradient
  shared    HCA attention of a batch whose sequences share a prefix of entries, each with entries of its own and a window
  weights   what every own entry received of the attention, added to the weights of the steps before
  evict     the entries with the largest weights kept, moved together, when a cache is cut down to a budget

Where `own` is false, run() computes them with elementary torch operations; where it is true, with the library's calls.
"""
import math

import torch

own = False

TWO_PI = 2.0 * math.pi
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One decode step of four sequences near 1M tokens: the query heads, the new K=V row and the indexer's heads. Latency.
        dict(name="rope_decode", op="rope", dtype="bf16", B=4, T=1, H=64, d=512, R=64, HI=16, DI=128, half=False, grad=False,
             factor=1.0, orig=0, pos=1048576, ragged=True),
        # The queries of a prefill chunk late in a 128K sequence. Bandwidth.
        dict(name="rope_chunk", op="rope", dtype="bf16", B=1, T=4096, H=64, d=512, R=64, HI=0, DI=0, half=False, grad=False,
             factor=1.0, orig=0, pos=126976, ragged=False),
        # The gradient for fp32 heads rotated over their whole width, half layout, scaled to sixteen times the trained length.
        dict(name="rope_grad_f32", op="rope", dtype="f32", B=2, T=777, H=16, d=128, R=128, HI=4, DI=64, half=True, grad=True,
             factor=16.0, orig=4096, pos=60000, ragged=True),
        # 32 conversations over one 1M-token document, a decode step each, some thousand own tokens, with sink and output rotation.
        dict(name="shared_1m", op="shared", dtype="bf16", B=32, T=1, H=64, d=512, Np=8192, rows=64, W=128, m=128, sink=True, R=64,
             ragged=True, evicted=False, padded=False),
        # Four sequences behind a 64K-token system prompt, just begun. Latency.
        dict(name="shared_64k", op="shared", dtype="bf16", B=4, T=1, H=64, d=512, Np=512, rows=16, W=128, m=128, sink=False, R=0,
             ragged=False, evicted=False, padded=False),
        # One of eight ranks that split the heads: 8 heads each, two tokens a step, a padded batch with evicted entries.
        dict(name="shared_heads8", op="shared", dtype="bf16", B=61, T=2, H=8, d=512, Np=4096, rows=200, W=128, m=128, sink=True, R=0,
             ragged=True, evicted=True, padded=True),
        # fp32, the small heads of the parity configuration.
        dict(name="shared_f32", op="shared", dtype="f32", B=3, T=1, H=16, d=128, Np=1000, rows=24, W=128, m=128, sink=False, R=0,
             ragged=True, evicted=False, padded=False),
        # The weights after a decode step of 32 sequences with full 1M-token caches of their own.
        dict(name="weights_1m", op="weights", dtype="bf16", B=32, T=1, H=64, d=512, Np=0, rows=8192, m=128, decay=1.0, ragged=False,
             evicted=False),
        # A small fp32 cache from which entries were evicted before, two tokens a step, older weights fading.
        dict(name="weights_f32", op="weights", dtype="f32", B=3, T=2, H=16, d=128, Np=64, rows=500, m=128, decay=0.98, ragged=True,
             evicted=True),
        # 32 full caches cut to half.
        dict(name="evict_1m", op="evict", dtype="bf16", B=32, d=512, rows=8192, budget=4096, first=4, recent=64, ragged=False,
             evicted=False),
        # A few small fp32 caches, ragged, cut for the second time. Latency.
        dict(name="evict_f32", op="evict", dtype="f32", B=4, d=128, rows=1000, budget=391, first=1, recent=32, ragged=True, evicted=True),
        # One sequence with a very long CSA cache cut to a quarter.
        dict(name="evict_long", op="evict", dtype="bf16", B=1, d=512, rows=262144, budget=65536, first=128, recent=4096, ragged=False,
             evicted=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "shared", "weights", "evict"])
    bf = rng.random() < 0.7
    dtype = "bf16" if bf else "f32"
    if op == "rope":
        d = 512 if bf else rng.choice([64, 128])
        R = rng.choice([64, 64, 128]) if bf else rng.choice([32, d // 2, d])
        H = rng.choice([8, 16, 64]) if bf else rng.choice([4, 16])
        B, HI = rng.choice([1, 2, 3, 4, 8]), rng.choice([0, 4, 16])
        T = _log_int(rng, 1, 4096 * 64 * 512 // (B * (H * d + d + HI * 128)) // (1 if bf else 4))
        scaled = rng.random() < 0.4
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, d=d, R=R, HI=HI, DI=128, half=rng.random() < 0.4,
                    grad=rng.random() < 0.4, factor=rng.choice([4.0, 16.0]) if scaled else 1.0, orig=rng.choice([0, 4096, 65536]) if scaled else 0,
                    pos=_log_int(rng, 1, 1 << 20), ragged=rng.random() < 0.5)
    if op == "shared":
        T = rng.choice([1, 1, 2, 3])
        if bf:
            H, d = rng.choice([8, 16, 32, 64, 64, 128]), 512
            B = _log_int(rng, 1, max(1, 2048 // (T * H)))
            Np = _log_int(rng, 1, 8192)
        else:
            H, d = rng.choice([4, 16]), rng.choice([64, 128])
            B = rng.randint(1, 6)
            Np = _log_int(rng, 1, 1500)
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, d=d, Np=Np, rows=_log_int(rng, 1, 256 if bf else 64), W=rng.choice([0, 64, 128, 128]),
                    m=128, sink=rng.random() < 0.5, R=rng.choice([0, 64]), ragged=rng.random() < 0.6, evicted=rng.random() < 0.4,
                    padded=rng.random() < 0.3)
    if op == "weights":
        T = rng.choice([1, 1, 2])
        if bf:
            H, d, B = rng.choice([8, 64, 64, 128]), 512, rng.randint(1, 32)
            rows = _log_int(rng, 1, min(32768, 262144 // (B * T * max(1, H // 64))))
        else:
            H, d, B = rng.choice([4, 16]), rng.choice([64, 128]), rng.randint(1, 6)
            rows = _log_int(rng, 1, 1500)
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, d=d, Np=rng.choice([0, 7, 512]), rows=rows, m=128, decay=rng.choice([1.0, 0.9, 0.0]),
                    ragged=rng.random() < 0.6, evicted=rng.random() < 0.4)
    B = rng.randint(1, 32)
    rows = _log_int(rng, 8, 262144 // B)
    budget = rng.randint(1, rows)
    first = rng.randint(0, min(8, budget))
    return dict(op=op, dtype=dtype, B=B, d=512 if bf else rng.choice([64, 128]), rows=rows, budget=budget, first=first,
                recent=rng.randint(0, min(128, budget - first)), ragged=rng.random() < 0.6, evicted=rng.random() < 0.4)


# ---------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cache(case, g):
    """Lengths, counts and, where entries were evicted before, the entry that every own slot holds."""
    B, T, rows, m, Np = case["B"], case["T"], case["rows"], case["m"], case["Np"]
    cnt = torch.full((B,), rows, dtype=torch.int64, device="cuda")
    if case["ragged"]:
        cnt = torch.randint(0, rows + 1, (B,), generator=g, device="cuda")
    total = cnt.clone()  # own entries that the sequence has had
    if case["evicted"]:
        total = cnt + torch.randint(0, rows + 1, (B,), generator=g, device="cuda")
    entry = None
    if case["evicted"]:  # the slots hold cnt of the total entries, in order: a random subset, the last entry among them
        u = torch.rand((B, 2 * rows), generator=g, device="cuda")
        pos = torch.arange(2 * rows, device="cuda")
        u = torch.where(pos == (total[:, None] - 1), -1.0, torch.where(pos < total[:, None], u, 2.0))
        rank = u.argsort(1).argsort(1)
        keep = torch.where(rank < cnt[:, None], pos, 4 * rows).sort(1).values[:, :rows]
        entry = (keep + Np).to(torch.int32).contiguous()
    lens = m * (Np + total) + torch.randint(T, m, (B,), generator=g, device="cuda")
    if case.get("padded") and B > 1:
        lens[B // 2] = 0
        cnt[B // 2] = 0
    return lens.contiguous(), cnt.to(torch.int32).contiguous(), entry


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    dt = DT[case["dtype"]]
    B, d = case["B"], case["d"]
    if case["op"] == "rope":
        T = case["T"]
        xs = [_normal((B, T, case["H"], d), dt, g), _normal((B, T, 1, d), dt, g)]
        if case["HI"] and case["R"] <= case["DI"]:
            xs.append(_normal((B, T, case["HI"], case["DI"]), dt, g))
        s["x"], s["y"] = xs, [torch.empty_like(x) for x in xs]
        start = torch.full((B, 1), case["pos"], dtype=torch.int64, device="cuda")
        if case["ragged"]:
            start = torch.randint(0, case["pos"] + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(T, device="cuda")).contiguous()
        return s
    if case["op"] == "evict":
        rows = case["rows"]
        s["cache"] = _normal((B, rows, d), dt, g)
        # attention gathers on few entries; many are equal, as they have received nothing worth counting
        w = torch.exp(2.0 * torch.randn((B, rows), generator=g, device="cuda"))
        s["weights"] = torch.where(torch.rand((B, rows), generator=g, device="cuda") < 0.3, (w * 4).round() / 4, w).contiguous()
        cnt = torch.full((B,), rows, device="cuda")
        if case["ragged"]:
            cnt = torch.randint(0, rows + 1, (B,), generator=g, device="cuda")
        s["count"] = cnt.to(torch.int32)
        s["entry"] = None
        if case["evicted"]:
            s["entry"] = torch.randint(1, 4, (B, rows), generator=g, device="cuda").cumsum(1).to(torch.int32).contiguous()
        k = case["budget"]
        s["out"] = dict(cache=torch.zeros((B, k, d), dtype=dt, device="cuda"), weights=torch.zeros((B, k), device="cuda"),
                        kept=torch.zeros((B, k), dtype=torch.int32, device="cuda"), count=torch.zeros((B,), dtype=torch.int32, device="cuda"),
                        entry=torch.zeros((B, k), dtype=torch.int32, device="cuda"))
        return s
    T, H, rows = case["T"], case["H"], case["rows"]
    s["q"] = _normal((B, T, H, d), dt, g)
    s["cache"] = _normal((B, rows, d), dt, g)
    s["lens"], s["count"], s["entry"] = _cache(case, g)
    s["ctx_len"] = case["m"] * (case["Np"] + (2 if case["evicted"] else 1) * rows + 1)
    if case["op"] == "shared":
        s["prefix"] = _normal((case["Np"], d), dt, g)
        s["ring"] = _normal((B, 256, d), dt, g)
        s["sink"] = torch.randn((H,), generator=g, device="cuda") if case["sink"] else None
        s["out"] = torch.empty((B, T, H, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((B, T, H), device="cuda")
        s["workspace"] = torch.empty(_shared_workspace(case), dtype=torch.uint8, device="cuda")
    else:
        s["weights"] = torch.rand((B, rows), generator=g, device="cuda") * 8
        logits = torch.bmm(s["q"].reshape(B, T * H, d).float(), s["cache"].float().transpose(1, 2)).view(B, T, H, rows) / math.sqrt(d)
        seen = _own_visible(s, case)[:, :, None, :]
        # the entries of the prefix and the window have a share of the whole too
        s["lse"] = torch.logaddexp(logits.masked_fill(~seen, -math.inf).logsumexp(-1), torch.full((), 2.0, device="cuda")).contiguous()
        s["out"] = torch.zeros((B, rows), device="cuda")
    return s


def _shared_workspace(case):
    """Scratch that a serving program sets aside once: generous for every shape of the cases."""
    q = case["B"] * case["T"]
    return 4 * (case["d"] + 2) * 64 * (160 * 4 + 4 * q * ((case["H"] + 63) // 64)) + (1 << 20)


# ---------------------------------------------------------------------- the operators, in plain form

def _frequencies(case):
    k = torch.arange(case["R"] // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * k / case["R"])
    if case["factor"] != 1.0:
        if case["orig"]:
            keep = ((case["orig"] * f / TWO_PI - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
            f = f * keep + f / case["factor"] * (1.0 - keep)
        else:
            f = f / case["factor"]
    return f


def _scale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["orig"] else 1.0


def _rope(x, case, positions):
    R, d = case["R"], x.shape[-1]
    ang = positions[:, :, None, None].double() * _frequencies(case)
    c, n = (ang.cos() * _scale(case)).float(), (ang.sin() * _scale(case) * (-1.0 if case["grad"] else 1.0)).float()
    xf = x.float()
    keep, r = xf[..., : d - R], xf[..., d - R:]
    if case["half"]:
        a, b = r[..., : R // 2], r[..., R // 2:]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    return torch.cat((keep, turned), -1).to(x.dtype)


def _query_pos(s, case):
    return s["lens"][:, None] - case["T"] + torch.arange(case["T"], device="cuda")


def _own_visible(s, case):
    """[B][T][rows]: whether query (b, j) sees own slot i."""
    slot = torch.arange(case["rows"], device="cuda")
    e = s["entry"].long() if s["entry"] is not None else (slot + case["Np"]).expand(case["B"], -1)
    t = _query_pos(s, case)
    return (slot < s["count"][:, None])[:, None, :] & (case["m"] * (e[:, None, :] + 1) <= t[:, :, None] + 1)


def _shared(s, case):
    B, T, H, d, Np, W = (case[k] for k in ("B", "T", "H", "d", "Np", "W"))
    q = s["q"].float()
    prefix = s["prefix"].float()
    cache = s["cache"].float()
    t = _query_pos(s, case)
    alive = (t >= 0)[:, :, None, None]
    lp = torch.matmul(q.reshape(-1, d), prefix.t()).view(B, T, H, Np)
    lo = torch.bmm(q.reshape(B, T * H, d), cache.transpose(1, 2)).view(B, T, H, -1)
    lo = lo.masked_fill(~_own_visible(s, case)[:, :, None, :], -math.inf)
    parts = [lp, lo]
    if W:
        p = t[:, :, None] - W + 1 + torch.arange(W, device="cuda")
        win = s["ring"][torch.arange(B, device="cuda")[:, None, None], p % s["ring"].shape[1]].float()
        parts.append(torch.matmul(q, win.transpose(2, 3)).masked_fill((p < 0)[:, :, None, :], -math.inf))
    logits = (torch.cat(parts, -1) / math.sqrt(d)).masked_fill(~alive, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = torch.where(alive, total + torch.exp(s["sink"][:, None] - top), total)
    o = torch.matmul(e[..., :Np].reshape(-1, Np), prefix).view(B, T, H, d)
    o = o + torch.bmm(e[..., Np: Np + case["rows"]].reshape(B, T * H, -1), cache).view(B, T, H, d)
    if W:
        o = o + torch.matmul(e[..., Np + case["rows"]:], win)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    if case["R"]:
        R = case["R"]
        k = torch.arange(R // 2, dtype=torch.float64, device="cuda")
        ang = -t[:, :, None, None].double() * 10000.0 ** (-2.0 * k / R)
        c, n = ang.cos().float(), ang.sin().float()
        a, b = o[..., d - R:: 2], o[..., d - R + 1:: 2]
        o = torch.cat((o[..., : d - R], torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)), -1)
    return {"out": o.to(s["q"].dtype), "lse": lse}


def _weights(s, case):
    B, T, H, d = (case[k] for k in ("B", "T", "H", "d"))
    logits = torch.bmm(s["q"].reshape(B, T * H, d).float(), s["cache"].float().transpose(1, 2)).view(B, T, H, -1) / math.sqrt(d)
    p = torch.exp(logits - s["lse"][..., None])
    got = torch.where(_own_visible(s, case), p.sum(2), 0.0).sum(1)
    held = torch.arange(case["rows"], device="cuda") < s["count"][:, None]
    return torch.where(held, s["weights"] * case["decay"] + got, 0.0)


def _evict(s, case):
    B, rows, k = case["B"], case["rows"], case["budget"]
    slot = torch.arange(rows, device="cuda")
    cnt = s["count"].long()[:, None]
    held = slot < cnt
    always = held & ((slot < case["first"]) | (slot >= cnt - case["recent"]))
    key = torch.where(always, math.inf, torch.where(held, s["weights"], -math.inf))
    order = key.argsort(dim=1, descending=True, stable=True)[:, :k]
    kept = torch.where(torch.arange(order.shape[1], device="cuda") < cnt, order, rows).sort(1).values
    there = kept < rows
    at = kept.clamp(max=rows - 1)
    row = torch.arange(B, device="cuda")[:, None]
    out = {"cache": torch.where(there[..., None], s["cache"][row, at], 0), "weights": torch.where(there, s["weights"][row, at], 0.0),
           "kept": torch.where(there, kept, -1).to(torch.int32), "count": there.sum(1).to(torch.int32)}
    if s["entry"] is not None:
        out["entry"] = torch.where(there, s["entry"][row, at], 0)
    return out


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "rope":
        return [_rope(x, case, s["positions"]) for x in s["x"]]
    return {"shared": _shared, "weights": _weights, "evict": _evict}[case["op"]](s, case)


def _own(s, case):
    import compressed_sparse_long_v4a_b200 as v4a
    if case["op"] == "rope":
        v4a.v4a_rope(list(zip(s["x"], s["y"])), rope_dims=case["R"], positions=s["positions"], rope_base=10000.0, half=case["half"],
                     inverse=case["grad"], factor=case["factor"], orig_ctx=case["orig"], out_scale=_scale(case))
        return s["y"]
    if case["op"] == "shared":
        v4a.v4a_hca_attend_shared(s["q"], s["prefix"], s["cache"], s["ring"] if case["W"] else None, s["out"], m=case["m"],
                                  window=case["W"], ctx_len=s["ctx_len"], ctx_lens=s["lens"], own_count=s["count"],
                                  own_entry=s["entry"], lse=s["lse"], sink=s["sink"], rope_dims=case["R"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "weights":
        v4a.v4a_attend_weights(s["q"], s["cache"], s["lse"], s["weights"], s["out"], n_prefix=case["Np"], m=case["m"],
                               ctx_len=s["ctx_len"], ctx_lens=s["lens"], own_count=s["count"], own_entry=s["entry"],
                               decay=case["decay"])
        return s["out"]
    o = s["out"]
    entry = s["entry"] is not None
    v4a.v4a_evict(s["cache"], s["weights"], o["cache"], o["weights"], o["kept"], o["count"], budget=case["budget"],
                  keep_first=case["first"], keep_recent=case["recent"], own_count=s["count"], own_entry=s["entry"],
                  entry_out=o["entry"] if entry else None)
    return {k: v for k, v in o.items() if k != "entry" or entry}


# ---------------------------------------------------------------------- what they cost at least

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, d = case["B"], case["d"]
    if case["op"] == "rope":
        n = case["H"] * d + d + (case["HI"] * case["DI"] if case["HI"] and case["R"] <= case["DI"] else 0)
        heads = case["H"] + 1 + case["HI"]
        return {"bytes": 2 * B * case["T"] * n * e + 8 * B * case["T"], "flops": 3 * B * case["T"] * heads * case["R"]}
    part = 0.5 if case["ragged"] else 1.0  # the mean of the counts
    if case["op"] == "evict":
        k = min(case["budget"], case["rows"] * part)
        return {"bytes": B * (4 * case["rows"] * part + k * (2 * d * e + 4 + 4 + (8 if case["evicted"] else 0))), "flops": 0}
    T, H = case["T"], case["H"]
    if case["op"] == "shared":
        keys = case["Np"] + case["rows"] * part + case["W"]
        rows = case["Np"] + B * (case["rows"] * part + case["W"])
        return {"bytes": rows * d * e + 2 * B * T * H * d * e + 4 * B * T * H, "flops": 4 * B * T * H * keys * d}
    n = B * case["rows"] * part
    return {"bytes": n * (d * e + 8) + B * T * H * (d * e + 4), "flops": 2 * n * T * H * d}


# ---------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    B, d = case["B"], case["d"]
    if case["op"] == "rope":
        R, got = case["R"], []
        freq = torch.tensor([_turn(case, i) for i in range(R // 2)], dtype=f8, device="cuda")
        w = torch.polar(torch.full_like(freq, _scale(case)).expand(*s["positions"].shape, -1),
                        (-1 if case["grad"] else 1) * s["positions"].to(f8)[..., None] * freq)[:, :, None, :]
        for x in s["x"]:
            y = x.to(f8).clone()
            tail = y[..., x.shape[-1] - R:]
            z = torch.complex(tail[..., : R // 2], tail[..., R // 2:]) if case["half"] else torch.view_as_complex(tail.reshape(*tail.shape[:-1], -1, 2).contiguous())
            z = z * w
            y[..., x.shape[-1] - R:] = torch.cat((z.real, z.imag), -1) if case["half"] else torch.view_as_real(z).flatten(-2)
            got.append(y)
        return got
    if case["op"] == "evict":
        out = _empty_evict(s, case)
        weights, counts = s["weights"].cpu().tolist(), s["count"].cpu().tolist()
        for b in range(B):
            n = counts[b]
            fixed = [i for i in range(n) if i < case["first"] or i >= n - case["recent"]]
            rest = sorted((i for i in range(case["first"], max(case["first"], n - case["recent"]))), key=lambda i: (-weights[b][i], i))
            keep = torch.tensor(sorted((fixed + rest)[: case["budget"]]), dtype=torch.long, device="cuda")
            out["cache"][b, : len(keep)] = s["cache"][b, keep].to(f8)
            out["weights"][b, : len(keep)] = s["weights"][b, keep].to(f8)
        return {"cache": out["cache"], "weights": out["weights"], "kept": None, "count": None}
    T, H, m, Np = case["T"], case["H"], case["m"], case["Np"]
    lens, counts = s["lens"].tolist(), s["count"].tolist()
    if case["op"] == "weights":
        got = torch.zeros((B, case["rows"]), dtype=f8, device="cuda")
        for b in range(B):
            n = counts[b]
            ent = s["entry"][b, :n].long() if s["entry"] is not None else torch.arange(n, device="cuda") + Np
            got[b, :n] = s["weights"][b, :n].to(f8) * case["decay"]
            for j in range(T):
                a = torch.einsum("hd,nd->hn", s["q"][b, j].to(f8), s["cache"][b, :n].to(f8)) * d ** -0.5
                p = (a - s["lse"][b, j].to(f8)[:, None]).exp() * ((ent + 1) * m <= lens[b] - T + j + 1)
                got[b, :n] += p.sum(0)
        return got
    out = torch.zeros((B, T, H, d), dtype=f8, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=f8, device="cuda")
    for b in range(B):
        n = counts[b]
        ent = s["entry"][b, :n].long() if s["entry"] is not None else torch.arange(n, device="cuda") + Np
        for j in range(T):
            t = lens[b] - T + j
            if t < 0:
                continue
            window = torch.arange(max(0, t - case["W"] + 1), t + 1, device="cuda") if case["W"] else torch.arange(0, device="cuda")
            kv = torch.cat((s["prefix"], s["cache"][b, :n][(ent + 1) * m <= t + 1], s["ring"][b, window % s["ring"].shape[1]])).to(f8)
            a = torch.einsum("hd,nd->hn", s["q"][b, j].to(f8), kv) * d ** -0.5
            if s["sink"] is not None:
                a = torch.cat((a, s["sink"].to(f8)[:, None]), 1)
            lse[b, j] = torch.logsumexp(a, 1)
            o = torch.einsum("hn,nd->hd", (a[:, : len(kv)] - lse[b, j][:, None]).exp(), kv)
            if case["R"]:
                R = case["R"]
                w = torch.polar(torch.ones(R // 2, dtype=f8, device="cuda"), -t * 10000.0 ** (-torch.arange(0, R, 2, dtype=f8, device="cuda") / R))
                z = torch.view_as_complex(o[:, d - R:].reshape(H, -1, 2).contiguous()) * w
                o = torch.cat((o[:, : d - R], torch.view_as_real(z).flatten(-2)), -1)
            out[b, j] = o
    return {"out": out, "lse": lse}


def _turn(case, i):
    """Radians per position of pair i."""
    f = math.exp(-math.log(10000.0) * 2 * i / case["R"])
    if case["factor"] == 1.0:
        return f
    if not case["orig"]:
        return f / case["factor"]
    turns = case["orig"] * f / TWO_PI
    ramp = min(1.0, max(0.0, (turns - 1.0) / 31.0))
    return f * ramp + f / case["factor"] * (1.0 - ramp)


def _empty_evict(s, case):
    return {"cache": torch.zeros((case["B"], case["budget"], case["d"]), dtype=torch.float64, device="cuda"),
            "weights": torch.zeros((case["B"], case["budget"]), dtype=torch.float64, device="cuda")}
