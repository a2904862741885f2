"""What the prompt, step and cache operators are timed on.

A case is one call of one operator at one size.  ``run`` computes it either in
a plain form (elementary torch operations in fp32, rounded once at the end) or,
where ``own`` is true, by the calls of block_sparse_attention_head_b200.
``exact`` computes the same from the definitions in 64 bits.

Operators (c = 1/sqrt(d), query head h reads key/value head h / G):
  prompt   packed sequences; query i of a sequence of n_q queries and n_k keys
           sees keys j <= i + n_k - n_q (all keys when not causal)
  weights  per key, the sum of its attention weights over all query rows and
           the G heads, added to what is there
  step     one query token per sequence; sees a prefix that the batch shares
           and the sequence's own cache; may add to the cache's key weights
  evict    keeps the most recent keys and those of the largest weights
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of short requests at once: latency
        dict(name="prompt tiny", op="prompt", nseq=3, q=37, k=37, hq=8, hkv=2, d=64, dtype="bf16", causal=True),
        # an ordinary prefill batch of requests of different lengths, 4 query heads to a key head
        dict(name="prompt packed", op="prompt", nseq=8, q=2048, k=2048, hq=32, hkv=8, d=128, dtype="bf16",
             causal=True),
        # one long document
        dict(name="prompt long", op="prompt", nseq=1, q=16384, k=16384, hq=16, hkv=4, d=128, dtype="bf16",
             causal=True),
        # the last chunk of long prompts against all their earlier keys, ungrouped heads
        dict(name="prompt chunk", op="prompt", nseq=4, q=257, k=8191, hq=40, hkv=40, d=128, dtype="fp16",
             causal=True),
        # attention mass of a prefill batch's keys
        dict(name="weights packed", op="weights", nseq=6, q=1000, k=1000, hq=32, hkv=8, d=128, dtype="bf16",
             causal=True),
        # attention mass that a long prompt's last 2048 queries give its keys
        dict(name="weights long", op="weights", nseq=1, q=2048, k=16384, hq=32, hkv=4, d=128, dtype="bf16",
             causal=True),
        # one request alone, short context, no shared prefix: latency
        dict(name="step one", op="step", batch=1, prefix=0, n=300, cap=512, hq=8, hkv=2, d=64, dtype="bf16",
             keep=False),
        # a batch behind one system prompt, its key weights kept for eviction
        dict(name="step batch", op="step", batch=32, prefix=4000, n=500, cap=1024, hq=32, hkv=8, d=128, dtype="bf16",
             keep=True),
        # many samples of one long document
        dict(name="step prefix", op="step", batch=128, prefix=32768, n=200, cap=256, hq=32, hkv=8, d=128,
             dtype="fp16", keep=False),
        # long private contexts, nothing shared
        dict(name="step own", op="step", batch=8, prefix=0, n=65000, cap=65536, hq=32, hkv=8, d=128, dtype="bf16",
             keep=True),
        # generation has filled its cache: 76 new keys in, back to 1024, in place
        dict(name="evict full", op="evict", batch=32, n=1100, cap=1100, budget=1024, recent=256, hkv=8, d=128,
             dtype="bf16", place=True),
        # long prompts' keys into small generation caches
        dict(name="evict prompt", op="evict", batch=8, n=16384, cap=16384, budget=2048, recent=128, hkv=8, d=128,
             dtype="bf16", place=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prompt", "weights", "step", "evict"])
    dtype, d = rng.choice(["bf16", "fp16"]), rng.choice([64, 128, 128])
    hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("prompt", "weights"):
        nseq = log(1, 16)
        k = log(1, 8192 if nseq <= 4 else 2048)
        q = k if rng.random() < 0.6 else max(1, k // rng.choice([2, 3, 7, 20]))
        while nseq * hkv * g * q * k > 16 * 16384 * 16384 // 4:
            hkv, g = max(1, hkv // 2), max(1, g // 2)
            if hkv * g == 1:
                break
        return dict(op=op, nseq=nseq, q=q, k=k, hq=hkv * g, hkv=hkv, d=d, dtype=dtype, causal=rng.random() < 0.8)
    if op == "step":
        batch = log(1, 128)
        prefix = 0 if rng.random() < 0.25 else log(1, 32768)
        n = log(1, max(2, min(32768, 400000 // (batch * hkv))))
        return dict(op=op, batch=batch, prefix=prefix, n=n, cap=n + rng.randint(0, 100), hq=hkv * g, hkv=hkv, d=d,
                    dtype=dtype, keep=rng.random() < 0.5)
    batch, place = log(1, 32), rng.random() < 0.5
    n = log(20, max(40, min(32768, 1000000 // (batch * hkv))))
    budget = max(2, n - rng.randint(1, max(2, n // 8))) if place else max(1, n // rng.choice([2, 3, 8]))
    return dict(op=op, batch=batch, n=n, cap=n if place else n + rng.randint(0, 50), budget=budget,
                recent=rng.randint(0, budget // 2), hkv=hkv, d=d, dtype=dtype, place=place)


def lengths(count, longest):
    """Lengths of `count` sequences: the first is the longest, the others spread over 30% to 100% of it."""
    return [longest if i == 0 else max(1, int(longest * (0.3 + 0.7 * ((i * 0.6180339887) % 1.0)))) for i in
            range(count)]


def prompt_lengths(case):
    ks = lengths(case["nseq"], case["k"])
    return ks if case["q"] == case["k"] else [min(case["q"], n) for n in ks], ks


def pairs(case):
    """Visible (query token, key) pairs."""
    n = 0
    for nq, nk in zip(*prompt_lengths(case)):
        n += nq * nk - (nq * (nq - 1) // 2 if case["causal"] else 0)
    return n


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, d = DTYPES[case["dtype"]], case["d"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    s = dict(case=case, scale=1.0 / math.sqrt(d))
    op = case["op"]
    if op in ("prompt", "weights"):
        qs, ks = prompt_lengths(case)
        tq, tk, hq, hkv = sum(qs), sum(ks), case["hq"], case["hkv"]
        s["cu_q"] = torch.tensor(np.cumsum([0] + qs), dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor(np.cumsum([0] + ks), dtype=torch.int32, device="cuda")
        s["most_q"], s["most_k"] = max(qs), max(ks)
        s["q"], s["k"], s["v"] = normal(tq, hq, d, scale=1.2), normal(tk, hkv, d, scale=1.2), normal(tk, hkv, d)
        if op == "weights":
            # the lse of these rows, as the prompt's attention returned it
            s["lse"] = plain_prompt(s)[1]
            del s["v"]
            s["weights"] = torch.rand(hkv, tk, generator=gen, device="cuda")
        return s
    if op == "step":
        b, p, cap, hq, hkv = case["batch"], case["prefix"], case["cap"], case["hq"], case["hkv"]
        s["q"] = normal(b, hq, d, scale=1.2)
        s["k_prefix"], s["v_prefix"] = normal(hkv, p, d, scale=1.2), normal(hkv, p, d)
        s["k_cache"], s["v_cache"] = normal(b, hkv, cap, d, scale=1.2), normal(b, hkv, cap, d)
        s["lens"] = torch.tensor(lengths(b, case["n"]), dtype=torch.int32, device="cuda")
        s["weights"] = torch.rand(b, hkv, cap, generator=gen, device="cuda") if case["keep"] else None
        return s
    b, cap, hkv, n = case["batch"], case["cap"], case["hkv"], case["n"]
    s["k_cache"], s["v_cache"] = normal(b, hkv, cap, d), normal(b, hkv, cap, d)
    # weights as they are met: a few large, many small, some equal
    w = torch.rand(b, hkv, cap, generator=gen, device="cuda") ** 6 * 40
    s["weights"] = torch.where(w < 0.01, torch.zeros_like(w), w)
    s["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").expand(b, hkv, cap).contiguous()
    if case["place"]:
        # generation fills slots budget .. n with new keys, then evicts
        fresh = n - case["budget"]
        s["lens"] = torch.full((b,), n, dtype=torch.int32, device="cuda")
        s["newest"] = torch.full((b,), n, dtype=torch.int32, device="cuda")
        s["new_k"], s["new_v"] = normal(b, hkv, fresh, d), normal(b, hkv, fresh, d)
        s["new_w"] = torch.rand(b, hkv, fresh, generator=gen, device="cuda")
        s["ages"] = torch.arange(fresh, dtype=torch.int32, device="cuda")
    else:
        s["lens"] = torch.tensor(lengths(b, n), dtype=torch.int32, device="cuda")
        m = case["budget"]
        s["out"] = (torch.zeros(b, hkv, m, d, dtype=dt, device="cuda"), torch.zeros(b, hkv, m, d, dtype=dt, device="cuda"),
                    torch.zeros(b, hkv, m, device="cuda"), torch.zeros(b, hkv, m, dtype=torch.int32, device="cuda"),
                    torch.zeros(b, dtype=torch.int32, device="cuda"))
    return s


# -------------------------------------------------------------- plain forms
def padded_rows(cu, most):
    """[sequences, most] row numbers of packed sequences (clamped into range) and which of them exist."""
    at = torch.arange(most, device=cu.device)
    n = (cu[1:] - cu[:-1]).long()
    rows = cu[:-1].long()[:, None] + torch.minimum(at[None], (n - 1).clamp(min=0)[:, None])
    return rows, at[None] < n[:, None], n


def packed_places(cu, total):
    """Sequence and place in it of each packed row."""
    t = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].long().contiguous(), t, right=True)
    return seq, t - cu[seq].long()


def plain_logits(s):
    """Masked logits [sequences, hkv, G, most_q, most_k] of padded sequences."""
    c = s["case"]
    rq, has_q, nq = padded_rows(s["cu_q"], s["most_q"])
    rk, has_k, nk = padded_rows(s["cu_k"], s["most_k"])
    q = s["q"].float()[rq].unflatten(2, (c["hkv"], c["hq"] // c["hkv"])).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[rk].permute(0, 2, 3, 1)[:, :, None]
    x = torch.matmul(q, k).mul_(s["scale"])
    at_k = torch.arange(s["most_k"], device=x.device)
    seen = has_q[:, :, None] & has_k[:, None, :]
    if c["causal"]:
        last = torch.arange(s["most_q"], device=x.device)[None] + (nk - nq)[:, None]
        seen = seen & (at_k[None, None] <= last[:, :, None])
    return x.masked_fill_(~seen[:, None, None], -math.inf), rk


def plain_prompt(s):
    c = s["case"]
    x, rk = plain_logits(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = s["v"].float()[rk].permute(0, 2, 1, 3)[:, :, None]
    o = torch.matmul(x, v).div_(torch.where(total == 0, torch.ones_like(total), total))
    lse = (total.log() + top)[..., 0]
    seq, at = packed_places(s["cu_q"], s["q"].shape[0])
    o = o.flatten(1, 2)[seq, :, at].to(s["q"].dtype)
    return o, lse.flatten(1, 2)[seq, :, at].t().contiguous()


def plain_weights(s):
    x, _ = plain_logits(s)
    rq, has_q, _ = padded_rows(s["cu_q"], s["most_q"])
    lse = s["lse"].t()[rq].unflatten(2, x.shape[1:3]).permute(0, 2, 3, 1)[..., None]
    lse = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    w = x.sub_(lse).exp_().sum((2, 3))
    seq, at = packed_places(s["cu_k"], s["k"].shape[0])
    return s["weights"].add_(w[seq, :, at].t())


def plain_step(s):
    c = s["case"]
    b, hkv, cap = c["batch"], c["hkv"], c["cap"]
    q = s["q"].float().unflatten(1, (hkv, c["hq"] // hkv))
    shared = torch.einsum("bhgd,hpd->bhgp", q, s["k_prefix"].float())
    private = torch.matmul(q, s["k_cache"].float().transpose(2, 3))
    live = torch.arange(cap, device=q.device)[None] < s["lens"][:, None]
    private = private.masked_fill_(~live[:, None, None], -math.inf)
    x = torch.cat([shared, private], -1).mul_(s["scale"])
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = (x - top).exp_()
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.einsum("bhgp,hpd->bhgd", p[..., :c["prefix"]], s["v_prefix"].float())
    o = o + torch.matmul(p[..., c["prefix"]:], s["v_cache"].float())
    out = o.flatten(1, 2).to(s["q"].dtype), (total.log() + top).flatten(1)
    if s["weights"] is None:
        return out
    return out + (s["weights"].add_(p[..., c["prefix"]:].sum(2)),)


def plain_kept(weights, pos, lens, budget, recent):
    """[B, hkv, budget] the slot that each slot of the evicted cache is filled from, and which of them are filled."""
    b, hkv, cap = weights.shape
    at = torch.arange(cap, device=weights.device)
    live = (at[None] < lens[:, None])[:, None]
    newest = torch.where(live, pos, torch.full_like(pos, -2 ** 31)).amax(-1, keepdim=True)
    rank = torch.where(torch.isnan(weights), torch.full_like(weights, -math.inf), weights + 0.0)
    order = torch.argsort(rank, dim=-1, descending=True, stable=True)
    safe = (live & (pos.long() > newest.long() - recent)).long()
    first = 2 - safe - live.long()  # 0 recent, 1 other live, 2 behind the end
    order = order.gather(2, torch.argsort(first.gather(2, order), dim=-1, stable=True))
    kept = torch.zeros_like(weights, dtype=torch.bool).scatter_(2, order[..., :budget], True) & live
    stays = kept & (at < budget)
    hole = live & ~kept & (at < budget)
    moves = kept & (at >= budget)
    # the n-th freed slot takes the n-th moving one
    movers = torch.argsort((~moves).long(), dim=-1, stable=True)
    nth = (hole.long().cumsum(-1) - 1).clamp(min=0)
    source = torch.where(hole, movers.gather(2, nth), at.expand_as(movers))[..., :budget]
    return source, (stays | hole)[..., :budget]


def plain_evict(s):
    c = s["case"]
    m, (k, v, w, pos) = c["budget"], (s["k_cache"], s["v_cache"], s["weights"], s["pos"])
    source, filled = plain_kept(w, pos, s["lens"], m, c["recent"])
    ko, vo, wo, po, lo = (k, v, w, pos, s["lens"]) if c["place"] else s["out"]
    wide = source[..., None].expand(-1, -1, -1, c["d"])
    ko[:, :, :m] = torch.where(filled[..., None], k.gather(2, wide), ko[:, :, :m])
    vo[:, :, :m] = torch.where(filled[..., None], v.gather(2, wide), vo[:, :, :m])
    wo[:, :, :m] = torch.where(filled, w.gather(2, source), wo[:, :, :m])
    po[:, :, :m] = torch.where(filled, pos.gather(2, source), po[:, :, :m])
    lo.copy_(s["lens"].clamp(max=m))
    return ko, vo, wo, po, lo


def append(s):
    """Generation's new keys enter the cache (both forms do this alike)."""
    m, n = s["case"]["budget"], s["case"]["n"]
    s["k_cache"][:, :, m:n] = s["new_k"]
    s["v_cache"][:, :, m:n] = s["new_v"]
    s["weights"][:, :, m:n] = s["new_w"]
    s["pos"][:, :, m:n] = s["newest"][:, None, None] + s["ages"]
    s["newest"] += n - m
    s["lens"].fill_(n)


# --------------------------------------------------------------------- pass
def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if op == "evict" and c["place"]:
        append(s)
    if own:
        import block_sparse_attention_head_b200 as ig

        if op == "prompt":
            return ig.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"])
        if op == "weights":
            return ig.key_weights(s["q"], s["k"], s["lse"], s["cu_q"], s["cu_k"], s["weights"], causal=c["causal"])
        if op == "step":
            out = ig.prefix_attention(s["q"], s["k_prefix"], s["v_prefix"], s["k_cache"], s["v_cache"], s["lens"],
                                      weights=s["weights"])
            return out if s["weights"] is None else out + (s["weights"],)
        return ig.evict(s["k_cache"], s["v_cache"], s["weights"], s["pos"], s["lens"], c["budget"], c["recent"],
                        out=None if c["place"] else s["out"])
    if op == "prompt":
        return plain_prompt(s)
    if op == "weights":
        return plain_weights(s)
    if op == "step":
        return plain_step(s)
    return plain_evict(s)


# --------------------------------------------------------------------- work
def work(case):
    op, d = case["op"], case["d"]
    if op in ("prompt", "weights"):
        qs, ks = prompt_lengths(case)
        tq, tk, hq, hkv = sum(qs), sum(ks), case["hq"], case["hkv"]
        if op == "prompt":
            return {"bytes": 2 * d * (2 * tq * hq + 2 * tk * hkv) + 4 * tq * hq, "flops": 4 * d * hq * pairs(case)}
        return {"bytes": 2 * d * (tq * hq + tk * hkv) + 4 * tq * hq + 8 * tk * hkv, "flops": 2 * d * hq * pairs(case)}
    if op == "step":
        b, hq, hkv, total = case["batch"], case["hq"], case["hkv"], sum(lengths(case["batch"], case["n"]))
        rows = hkv * (case["prefix"] + total)
        return {"bytes": 4 * d * rows + 4 * d * b * hq + 4 * b * hq + (8 * hkv * total if case["keep"] else 0),
                "flops": 4 * d * hq * (b * case["prefix"] + total)}
    b, hkv, n, m = case["batch"], case["hkv"], case["n"], case["budget"]
    row = 4 * d + 8
    if case["place"]:
        # new rows in, ranks of all keys, and at most as many rows moved as are new
        return {"bytes": b * hkv * (2 * (n - m) * row + 8 * n + 2 * (n - m) * row), "flops": 0}
    ns = lengths(b, n)
    return {"bytes": hkv * sum(8 * x + 2 * min(x, m) * row for x in ns), "flops": 0}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "weights"):
        qs, ks = prompt_lengths(case)
        g = case["hq"] // case["hkv"]
        q, k, v = (s[n].double() for n in ("q", "k", "v" if op == "prompt" else "k"))
        o, lse = torch.zeros_like(q), torch.zeros(case["hq"], q.shape[0], dtype=torch.float64, device="cuda")
        w = s["weights"].double() if op == "weights" else None
        i = j = 0
        for nq, nk in zip(qs, ks):
            for h in range(case["hq"]):
                x = q[i:i + nq, h] @ k[j:j + nk, h // g].t() * s["scale"]
                if case["causal"]:
                    x.masked_fill_(torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1), -math.inf)
                if op == "weights":
                    w[h // g, j:j + nk] += torch.exp(x - s["lse"][h, i:i + nq, None].double()).sum(0)
                else:
                    lse[h, i:i + nq] = torch.logsumexp(x, 1)
                    o[i:i + nq, h] = torch.softmax(x, 1) @ v[j:j + nk, h // g]
            i, j = i + nq, j + nk
        return w if op == "weights" else (o, lse)
    if op == "step":
        p, g = case["prefix"], case["hq"] // case["hkv"]
        o = torch.zeros(case["batch"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
        lse = torch.zeros(case["batch"], case["hq"], dtype=torch.float64, device="cuda")
        w = s["weights"].double() if case["keep"] else None
        kp, vp = s["k_prefix"].double(), s["v_prefix"].double()
        for b, n in enumerate(lengths(case["batch"], case["n"])):
            k = torch.cat([kp, s["k_cache"][b, :, :n].double()], 1)
            v = torch.cat([vp, s["v_cache"][b, :, :n].double()], 1)
            q = s["q"][b].double().reshape(case["hkv"], g, case["d"])
            x = q @ k.transpose(1, 2) * s["scale"]
            a = torch.softmax(x, -1)
            o[b], lse[b] = (a @ v).reshape(-1, case["d"]), torch.logsumexp(x, -1).reshape(-1)
            if w is not None:
                w[b, :, :n] += a[..., p:].sum(1)
        return (o, lse) if w is None else (o, lse, w)
    if case["place"]:
        append(s)
    m, ins = case["budget"], (s["k_cache"], s["v_cache"], s["weights"], s["pos"])
    outs = ins if case["place"] else s["out"]
    done = [x.cpu().numpy() if x.dtype == torch.int32 else x.double().cpu().numpy() for x in outs[:4]]
    have = [x.cpu().numpy() if x.dtype == torch.int32 else x.double().cpu().numpy() for x in ins]
    ns = [int(n) for n in s["lens"]]
    for b, n in enumerate(ns):
        for h in range(case["hkv"]):
            w, pos = have[2][b, h, :n], have[3][b, h, :n]
            safe = pos > pos.max() - case["recent"]
            kept = np.lexsort((np.arange(n), -w, ~safe))[:m]
            freed = sorted(set(range(min(n, m))) - set(kept.tolist()))
            for x, y in zip(have, done):
                y[b, h, :min(n, m)] = x[b, h, :min(n, m)]
                y[b, h, freed] = x[b, h, sorted(kept[kept >= m])]
    return tuple(done) + (np.minimum(ns, m).astype(np.int32),)
