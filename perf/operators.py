"""What the framework's attention operators for language models are measured on: attention with
modified scores (tanh cap, distance bias, document and prefix masks), decode attention over a
paged key-value cache, appending to that cache, and eviction from it by accumulated weight.

``run`` computes an operator with elementary torch operations in 32 bits (``own`` false) or
calls the framework (``own`` true); ``exact`` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the grouped-head causal decoder at 8K tokens, scores capped as capped-logit decoders do
        scored("scored_decoder8k_cap", B=1, Hq=32, Hkv=8, Nq=8192, Nk=8192, d=128, dtype="bf16", layout="NHD",
               causal=True, cap=50.0),
        # the 4K self-attention shape, every key visible, biased by distance
        scored("scored_4k_bias", B=2, Hq=8, Hkv=8, Nq=4096, Nk=4096, d=128, dtype="fp16", layout="HND", bias=True),
        # a row of packed documents of ragged lengths with padding at its end, as a packed batch has
        scored("scored_packed_docs", B=1, Hq=8, Hkv=8, Nq=16383, Nk=16383, d=64, dtype="bf16", layout="NHD",
               causal=True, docs=14, pad=250, lens_seed=3),
        # the next chunk of a prompt against what came before it: few rows, many keys
        scored("scored_chunk", B=1, Hq=32, Hkv=8, Nq=100, Nk=20001, d=128, dtype="bf16", layout="HND",
               causal=True, offset=19901, bias=True),
        # a small batch of prefix-masked prompts with an odd head_dim, cap and bias together
        scored("scored_prefix_small", B=4, Hq=8, Hkv=2, Nq=257, Nk=257, d=72, dtype="fp16", layout="HND",
               causal=True, prefix=True, cap=30.0, bias=True, lens_seed=5),
        # one user, a short conversation: latency counts
        paged("paged_one", B=1, Hq=32, Hkv=8, lo=1000, hi=1000, d=128, dtype="bf16", page=16),
        # a serving batch of very different lengths, capped scores
        paged("paged_ragged32", B=32, Hq=32, Hkv=8, lo=128, hi=32768, d=128, dtype="bf16", page=64, cap=50.0,
              layout="NHD", lens_seed=7),
        # two long contexts, one key-value head per query head, weights accumulated for eviction
        paged("paged_long_mass", B=2, Hq=32, Hkv=32, lo=50001, hi=60001, d=64, dtype="fp16", page=128, bias=True,
              mass=True, lens_seed=9),
        # one token of every sequence of a decode step
        append("append_step", B=64, new=1, Hkv=8, old=2000, d=128, dtype="bf16", page=16, mass=True),
        # the prompts of a batch
        append("append_prompts", B=16, new=4096, Hkv=8, old=0, d=128, dtype="bf16", page=64, layout="NHD",
               lens_seed=11),
        # a cache a few tokens over its budget
        evict("evict_step", B=16, Hkv=8, lo=2049, hi=2112, budget=2048, sink=4, recent=128, d=128, dtype="bf16",
              page=16, lens_seed=13),
        # long prompts cut down to the budget
        evict("evict_prompts", B=8, Hkv=8, lo=6000, hi=32768, budget=4096, sink=4, recent=512, d=128,
              dtype="bf16", page=64, layout="NHD", lens_seed=15),
    ]


def scored(name, **kw):
    c = dict(op="scored", causal=False, cap=0.0, bias=False, docs=0, pad=0, prefix=False, offset=0, lens_seed=0)
    return dict(c, **kw, **({"name": name} if name else {}))


def paged(name, **kw):
    c = dict(op="paged", layout="HND", cap=0.0, bias=False, mass=False, lens_seed=0)
    return dict(c, **kw, **({"name": name} if name else {}))


def append(name, **kw):
    c = dict(op="append", layout="HND", mass=False, lens_seed=0)
    return dict(c, **kw, **({"name": name} if name else {}))


def evict(name, **kw):
    return dict(dict(op="evict", layout="HND", lens_seed=0), **kw, **({"name": name} if name else {}))


def log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["scored", "scored", "scored", "paged", "paged", "paged", "append", "evict"])
    d = rng.choice([64, 64, 128, 128, 128, 32, 72, 80, 96, 120])
    dtype, layout, seed = rng.choice(["fp16", "bf16"]), rng.choice(["HND", "NHD"]), rng.randrange(1 << 20)
    page = rng.choice([8, 16, 16, 32, 48, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    if op == "scored":
        hq = hkv * rng.choice([1, 2, 4, 4])
        nq = log_int(rng, 1, 8192)
        nk = nq if rng.random() < 0.5 else log_int(rng, nq, 24000)
        b = log_int(rng, 1, 8)
        while b > 1 and b * hq * nq * nk > 32 * 4096 * 8192:
            b -= 1
        while b * hq * nq * nk > 32 * 4096 * 8192:
            nq = max(1, nq // 2)
            nk = max(nq, nk - nk // 3)
        causal = rng.random() < 0.7
        docs = rng.randrange(2, 20) if nq == nk and nq >= 64 and rng.random() < 0.4 else 0
        return scored("", B=b, Hq=hq, Hkv=hkv, Nq=nq, Nk=nk, d=d, dtype=dtype, layout=layout, causal=causal,
                      cap=rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]), bias=rng.random() < 0.4, docs=docs,
                      pad=nq // 20 if docs else 0, prefix=causal and rng.random() < 0.3,
                      offset=nk - nq if causal else 0, lens_seed=seed)
    if op == "paged":
        hi = log_int(rng, 20, 60000)
        lo = max(1, rng.choice([hi, hi // 2, hi // 50]))
        b = log_int(rng, 1, 64)
        while b > 1 and b * hkv * hi * d > 32 * 8 * 20000 * 128:
            b -= 1
        return paged("", B=b, Hq=hkv * rng.choice([1, 2, 4, 8, 7, 16]), Hkv=hkv, lo=lo, hi=hi, d=d, dtype=dtype,
                     page=page, layout=layout, cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.3,
                     mass=rng.random() < 0.3, lens_seed=seed)
    if op == "append":
        b = log_int(rng, 1, 64)
        return append("", B=b, new=log_int(rng, 1, max(1, 60000 // b)), Hkv=hkv, old=rng.choice([0, 77, 1000]), d=d,
                      dtype=dtype, page=page, layout=layout, mass=rng.random() < 0.5, lens_seed=seed)
    hi = log_int(rng, 300, 40000)
    budget = log_int(rng, 64, max(65, hi - hi // 8))
    b = log_int(rng, 1, 16)
    while b > 1 and b * hi > 8 * 32768:
        b -= 1
    return evict("", B=b, Hkv=hkv, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, budget=budget,
                 sink=rng.choice([0, 4]), recent=budget // rng.choice([2, 4, 16]), d=d, dtype=dtype, page=page,
                 layout=layout, lens_seed=seed)


# ------------------------------------------------------- what a case says apart from the values
def lengths(c):
    """Lengths of the sequences in a cache case (new tokens for append), the largest one `hi`."""
    r = random.Random(c["lens_seed"])
    if c["op"] == "append":
        return [c["new"]] + [r.randint(max(1, c["new"] // 4), c["new"]) for _ in range(c["B"] - 1)]
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["B"] - 1)]


def document_ids(c, b):
    """Ids of one row of packed documents: ragged lengths, -1 where the row is padded."""
    r = random.Random(c["lens_seed"] * 1000 + b)
    n = c["Nq"] - c["pad"]
    cuts = sorted(r.randrange(n + 1) for _ in range(c["docs"] - 1))
    ids = []
    for i, (x, y) in enumerate(zip([0] + cuts, cuts + [n])):
        ids += [i] * (y - x)
    return ids + [-1] * c["pad"]


def prefix_lengths(c):
    r = random.Random(c["lens_seed"] + 1)
    return [r.randint(0, c["Nk"]) for _ in range(c["B"])]


def pairs(c):
    """Visible (query, key) pairs of one head, over the batch."""
    total = 0
    for b in range(c["B"]):
        pre = prefix_lengths(c)[b] if c["prefix"] else 0
        runs = [(0, c["Nq"], 0, c["Nk"])]
        if c["docs"]:
            ids, runs, at = document_ids(c, b), [], 0
            while at < len(ids):
                end = at
                while end < len(ids) and ids[end] == ids[at]:
                    end += 1
                if ids[at] >= 0:
                    runs.append((at, end, at, end))
                at = end
        for q0, q1, k0, k1 in runs:
            if not c["causal"]:
                total += (q1 - q0) * (k1 - k0)
            else:
                total += sum(max(0, min(k1, max(i + c["offset"] + 1, pre)) - k0) for i in range(q0, q1))
    return total


def work(c):
    e = 2
    if c["op"] == "scored":
        rows, keys = c["B"] * c["Nq"], c["B"] * c["Nk"]
        by = 2 * rows * c["Hq"] * c["d"] * e + 2 * keys * c["Hkv"] * c["d"] * e + 4 * rows * c["Hq"]
        return {"bytes": by, "flops": 4 * c["Hq"] * c["d"] * pairs(c)}
    n = sum(lengths(c))
    if c["op"] == "paged":
        by = 2 * n * c["Hkv"] * c["d"] * e + 2 * c["B"] * c["Hq"] * c["d"] * e + (8 * n * c["Hkv"] if c["mass"] else 0)
        return {"bytes": by, "flops": 4 * n * c["Hq"] * c["d"]}
    if c["op"] == "append":
        return {"bytes": 4 * n * c["Hkv"] * c["d"] * e + (8 * n * c["Hkv"] if c["mass"] else 0), "flops": 0}
    # eviction: masses and positions are read; of the freely chosen tokens, the share behind the budget moves
    by = 0.0
    for m in lengths(c):
        by += 8 * m * c["Hkv"]
        if m > c["budget"]:
            free, others = c["budget"] - c["sink"] - c["recent"], m - c["sink"] - c["recent"]
            behind = min(c["recent"], m - c["budget"])
            moved = behind + free * max(0, m - c["budget"] - c["recent"]) / max(1, others)
            by += moved * c["Hkv"] * (4 * c["d"] * e + 16)
    return {"bytes": by, "flops": 0}


# ------------------------------------------------------------------------------------ inputs
def normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def slopes_of(c, heads):
    """A geometric row of slopes, as distance-biased attention uses."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32, device=DEV)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"case": c}
    if c["op"] == "scored":
        hnd = c["layout"] == "HND"
        shape = lambda h, n: (c["B"], h, n, c["d"]) if hnd else (c["B"], n, h, c["d"])  # noqa: E731
        s["q"] = normal(g, shape(c["Hq"], c["Nq"]), dt, 2.0)
        offset = torch.randn((c["Hkv"], 1, c["d"]) if hnd else (c["Hkv"], c["d"]), generator=g, device=DEV)
        s["k"] = (torch.randn(shape(c["Hkv"], c["Nk"]), generator=g, device=DEV) + offset).to(dt)
        s["v"] = normal(g, shape(c["Hkv"], c["Nk"]), dt)
        s["slopes"] = slopes_of(c, c["Hq"]) if c["bias"] else None
        s["doc_ids"] = ints([document_ids(c, b) for b in range(c["B"])]) if c["docs"] else None
        s["prefix"] = ints(prefix_lengths(c)) if c["prefix"] else None
        return s
    lens = lengths(c)
    old = c["old"] if c["op"] == "append" else 0
    need = [-(-(n + old) // c["page"]) for n in lens]
    width, pages = max(need), sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table, at = torch.zeros((c["B"], width), dtype=torch.int32, device=DEV), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    hnd = c["layout"] == "HND"
    shape = (pages, c["Hkv"], c["page"], c["d"]) if hnd else (pages, c["page"], c["Hkv"], c["d"])
    plane = (pages, c["Hkv"], c["page"])
    if c["op"] == "append":
        s["kc"], s["vc"] = torch.zeros(shape, dtype=dt, device=DEV), torch.zeros(shape, dtype=dt, device=DEV)
        s["k"], s["v"] = (normal(g, (sum(lens), c["Hkv"], c["d"]), dt) for _ in "kv")
        s["lens"] = torch.full((c["B"],), old, dtype=torch.int32, device=DEV)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = ints(cu)
        s["step"] = c["new"] == 1
        # the sequence of every new token and its place there, which the plain form indexes with
        s["seq"] = torch.repeat_interleave(torch.arange(c["B"], device=DEV), ints(lens).long())
        s["mass"] = torch.full(plane, 7.0, device=DEV) if c["mass"] else None
        s["kpos"] = torch.full(plane, -1, dtype=torch.int32, device=DEV) if c["mass"] else None
        return s
    s["kc"], s["vc"] = normal(g, shape, dt), normal(g, shape, dt)
    s["lens"], s["max_len"] = ints(lens), c["hi"]
    if c["op"] == "paged":
        s["q"] = normal(g, (c["B"], c["Hq"], c["d"]), dt, 2.0)
        s["slopes"] = slopes_of(c, c["Hq"]) if c["bias"] else None
        s["mass"] = torch.rand(plane, generator=g, device=DEV) if c["mass"] else None
        return s
    # masses as accumulated softmax weights are: heavy-tailed, many exact zeros
    m = torch.exp(2.0 * torch.randn(plane, generator=g, device=DEV))
    s["mass0"] = torch.where(torch.rand(plane, generator=g, device=DEV) < 0.0625, 0.0, m)
    slot = torch.arange(width * c["page"], device=DEV, dtype=torch.int32).view(width, c["page"])
    kpos = torch.zeros(plane, dtype=torch.int32, device=DEV)
    for b, n in enumerate(need):
        kpos[table[b, :n].long()] = slot[:n, None, :].expand(n, c["Hkv"], c["page"])
    s["kpos0"] = kpos
    return s


# ------------------------------------------------------------------------------------ passes
def run(s):
    c = s["case"]
    if c["op"] == "scored":
        return run_scored(s, c)
    if c["op"] == "paged":
        return run_paged(s, c)
    if c["op"] == "append":
        return run_append(s, c)
    return run_evict(s, c)


def run_scored(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        out, lse = qa.scored_attn(s["q"], s["k"], s["v"], tensor_layout=c["layout"], is_causal=c["causal"],
                                  softcap=c["cap"], slopes=s["slopes"], prefix_lens=s["prefix"],
                                  doc_ids=s["doc_ids"], q_offset=c["offset"], return_lse=True)
        return {"out": out, "lse": lse}
    q, k, v = (t if c["layout"] == "HND" else t.transpose(1, 2) for t in (s["q"], s["k"], s["v"]))
    B, Hq, Nq, d = q.shape
    Hkv, Nk, g = k.shape[1], k.shape[2], Hq // k.shape[1]
    t = torch.matmul(q.float().reshape(B, Hkv, g * Nq, d), k.float().transpose(2, 3)).view(B, Hkv, g, Nq, Nk)
    t *= 1.0 / math.sqrt(d)
    if c["cap"]:
        t /= c["cap"]
        t.tanh_()
        t *= c["cap"]
    i = torch.arange(Nq, device=DEV)[:, None] + c["offset"]
    j = torch.arange(Nk, device=DEV)[None, :]
    if c["bias"]:
        t -= s["slopes"].view(1, Hkv, g, 1, 1) * (i - j).abs().float()
    seen = torch.ones((B, Nq, Nk), dtype=torch.bool, device=DEV)
    if c["causal"]:
        seen &= j <= i
        if c["prefix"]:
            seen |= j < s["prefix"].view(B, 1, 1)
    if c["docs"]:
        ids = s["doc_ids"]
        seen &= (ids[:, :, None] == ids[:, None, :]) & (ids[:, None, :] >= 0)
    t.masked_fill_(~seen[:, None, None], -math.inf)
    m = t.amax(-1, keepdim=True)
    any_seen = m > -math.inf
    t -= torch.where(any_seen, m, 0.0)
    t.exp_()
    total = t.sum(-1, keepdim=True)
    o = torch.matmul(t.view(B, Hkv, g * Nq, Nk), v.float()).view(B, Hkv, g, Nq, d)
    o = torch.where(any_seen, o / total, 0.0).view(B, Hq, Nq, d).to(s["q"].dtype)
    lse = torch.where(any_seen, m + torch.log(total), -math.inf).view(B, Hq, Nq)
    return {"out": o if c["layout"] == "HND" else o.transpose(1, 2).contiguous(), "lse": lse}


def gathered(cache, table, layout):
    """[B, Hkv, tokens, d] of the pages of a table, or [B, Hkv, tokens] of a plane's."""
    x = cache[table.long()]
    if x.dim() == 4:
        return x.transpose(1, 2).flatten(2, 3)
    return (x.transpose(1, 2) if layout == "HND" else x.permute(0, 3, 1, 2, 4)).flatten(2, 3)


def run_paged(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        out, lse = qa.paged_attn(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["max_len"],
                                 tensor_layout=c["layout"], softcap=c["cap"], slopes=s["slopes"], mass=s["mass"],
                                 return_lse=True)
        return {"out": out, "lse": lse, "mass": s["mass"]}
    k, v = (gathered(x, s["table"], c["layout"]).float() for x in (s["kc"], s["vc"]))
    B, Hkv, L, d = k.shape
    g = c["Hq"] // Hkv
    t = torch.matmul(s["q"].float().view(B, Hkv, g, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if c["cap"]:
        t = c["cap"] * torch.tanh(t / c["cap"])
    j = torch.arange(L, device=DEV)
    if c["bias"]:
        t = t - s["slopes"].view(1, Hkv, g, 1) * (s["lens"][:, None] - 1 - j).abs().float().view(B, 1, 1, L)
    seen = (j < s["lens"][:, None]).view(B, 1, 1, L)
    t = torch.where(seen, t, -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - m)
    total = p.sum(-1, keepdim=True)
    out = (torch.matmul(p, v) / total).view(B, c["Hq"], d).to(s["q"].dtype)
    if c["mass"]:
        add = (p / total).sum(2).view(B, Hkv, -1, c["page"]).transpose(1, 2)
        at = s["table"].long().flatten()
        s["mass"].index_put_((at,), add.reshape(at.numel(), Hkv, c["page"]), accumulate=True)
    return {"out": out, "lse": (m + torch.log(total)).view(B, c["Hq"]), "mass": s["mass"]}


def run_append(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        qa.paged_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                        cu_seqlens=None if s["step"] else s["cu"], tensor_layout=c["layout"], mass=s["mass"],
                        key_positions=s["kpos"])
        return {"k": s["kc"], "v": s["vc"], "mass": s["mass"], "positions": s["kpos"]}
    slot = torch.arange(s["seq"].numel(), device=DEV) - s["cu"].long()[s["seq"]] + s["lens"].long()[s["seq"]]
    page, at = s["table"].long()[s["seq"], slot // c["page"]], slot % c["page"]
    if c["layout"] == "HND":
        s["kc"][page, :, at], s["vc"][page, :, at] = s["k"], s["v"]
    else:
        s["kc"][page, at], s["vc"][page, at] = s["k"], s["v"]
    if c["mass"]:
        s["mass"][page, :, at] = 0.0
        s["kpos"][page, :, at] = slot.to(torch.int32)[:, None].expand(-1, c["Hkv"])
    return {"k": s["kc"], "v": s["vc"], "mass": s["mass"], "positions": s["kpos"]}


def run_evict(s, c):
    # the planes are this pass's own, so that every pass finds the same tokens to drop
    mass, kpos = s["mass0"].clone(), s["kpos0"].clone()
    if own:
        import quantized_attention_mean_gb300 as qa
        lens = qa.paged_evict(s["kc"], s["vc"], mass, kpos, s["table"], s["lens"], c["budget"], s["max_len"],
                              sink=c["sink"], recent=c["recent"], tensor_layout=c["layout"])
        return {"lens": lens, "k": s["kc"], "v": s["vc"], "mass": mass, "positions": kpos}
    w, p = gathered(mass, s["table"], ""), gathered(kpos, s["table"], "")
    B, Hkv, L = w.shape
    j = torch.arange(L, device=DEV).view(1, 1, L)
    n = s["lens"].view(B, 1, 1).long()
    held = j < n
    last = torch.where(held, p, -1).amax(-1, keepdim=True)
    guarded = (p < c["sink"]) | (p > last - c["recent"])
    key = torch.where(guarded, math.inf, torch.where(torch.isnan(w), -math.inf, w))
    # held tokens before the places behind the last one, then the largest weight, then the lowest slot
    order = torch.sort(torch.where(held, key.double(), math.nan).nan_to_num(nan=-1e300, posinf=1e301, neginf=-1e299),
                       dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand(B, Hkv, L).contiguous())
    keep = held & (rank < torch.clamp(n, max=c["budget"]))
    over = n > c["budget"]
    hole, mover = over & (j < c["budget"]) & ~keep, over & (j >= c["budget"]) & keep
    b, h, to = torch.nonzero(hole, as_tuple=True)
    _, _, of = torch.nonzero(mover, as_tuple=True)
    table = s["table"].long()
    tp, ts, fp, fs = table[b, to // c["page"]], to % c["page"], table[b, of // c["page"]], of % c["page"]
    mass[tp, h, ts], kpos[tp, h, ts] = mass[fp, h, fs], kpos[fp, h, fs]
    if c["layout"] == "HND":
        s["kc"][tp, h, ts], s["vc"][tp, h, ts] = s["kc"][fp, h, fs], s["vc"][fp, h, fs]
    else:
        s["kc"][tp, ts, h], s["vc"][tp, ts, h] = s["kc"][fp, fs, h], s["vc"][fp, fs, h]
    return {"lens": torch.clamp(s["lens"], max=c["budget"]), "k": s["kc"], "v": s["vc"], "mass": mass,
            "positions": kpos}


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"scored": exact_scored, "paged": exact_paged, "append": exact_append, "evict": exact_evict}[c["op"]](s, c)


def softmax64(t, seen, v):
    """Rows of softmax(t over seen) v and their log-sum-exp, in 64 bits; nothing seen: 0 and -inf."""
    t = torch.where(seen, t, -math.inf)
    lse = torch.logsumexp(t, -1)
    p = torch.exp(t - torch.where(lse > -math.inf, lse, 0.0)[..., None])
    return p @ v, lse, p


def exact_scored(s, c):
    nq, nk, g = c["Nq"], c["Nk"], c["Hq"] // c["Hkv"]
    head = lambda t, b, h: (t[b, h] if c["layout"] == "HND" else t[b, :, h]).double()  # noqa: E731
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros((c["B"], c["Hq"], nq), dtype=torch.float64, device=DEV)
    place = torch.arange(nk, device=DEV)
    rows = max(1, (1 << 27) // nk)
    for b in range(c["B"]):
        ids = torch.tensor(document_ids(c, b), device=DEV) if c["docs"] else None
        pre = prefix_lengths(c)[b] if c["prefix"] else 0
        for h in range(c["Hq"]):
            q, k, v = head(s["q"], b, h), head(s["k"], b, h // g), head(s["v"], b, h // g)
            for r in range(0, nq, rows):
                pos = torch.arange(r, min(nq, r + rows), device=DEV)[:, None] + c["offset"]
                t = q[r:r + rows] @ k.T / math.sqrt(c["d"])
                if c["cap"]:
                    t = torch.tanh(t / c["cap"]) * c["cap"]
                if c["bias"]:
                    t = t - float(s["slopes"][h]) * (pos - place).abs()
                seen = torch.ones_like(t, dtype=torch.bool)
                if c["causal"]:
                    seen = (place <= pos) | (place < pre)
                if c["docs"]:
                    mine = ids[r:r + rows, None]
                    seen = seen & (mine == ids) & (mine >= 0)
                o, l, _ = softmax64(t, seen, v)
                if c["layout"] == "HND":
                    out[b, h, r:r + rows] = o
                else:
                    out[b, r:r + rows, h] = o
                lse[b, h, r:r + rows] = l
    return {"out": out, "lse": lse}


def token_pages(s, c, b, n):
    slot = torch.arange(n, device=DEV)
    return s["table"][b].long()[slot // c["page"]], slot % c["page"]


def exact_paged(s, c):
    g = c["Hq"] // c["Hkv"]
    out = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((c["B"], c["Hq"]), dtype=torch.float64, device=DEV)
    mass = s["mass"].double() if c["mass"] else None
    for b, n in enumerate(lengths(c)):
        page, at = token_pages(s, c, b, n)
        for h in range(c["Hkv"]):
            k, v = ((x[page, h, at] if c["layout"] == "HND" else x[page, at, h]).double() for x in (s["kc"], s["vc"]))
            t = s["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(c["d"])
            if c["cap"]:
                t = torch.tanh(t / c["cap"]) * c["cap"]
            if c["bias"]:
                t = t - s["slopes"][h * g:(h + 1) * g, None].double() * torch.arange(n - 1, -1, -1, device=DEV)
            o, l, p = softmax64(t, torch.ones_like(t, dtype=torch.bool), v)
            out[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = o, l
            if c["mass"]:
                mass[page, h, at] += p.sum(0)
    return {"out": out, "lse": lse, "mass": mass}


def exact_append(s, c):
    k, v = s["kc"].double(), s["vc"].double()
    mass = s["mass"].double() if c["mass"] else None
    first = 0
    for b, n in enumerate(lengths(c)):
        page, at = (x[c["old"]:] for x in token_pages(s, c, b, c["old"] + n))
        for to, of in ((k, s["k"]), (v, s["v"])):
            if c["layout"] == "HND":
                to[page, :, at] = of[first:first + n].double()
            else:
                to[page, at] = of[first:first + n].double()
        if c["mass"]:
            mass[page, :, at] = 0.0
        first += n
    return {"k": k, "v": v, "mass": mass, "positions": None}


def exact_evict(s, c):
    k, v, mass = s["kc"].clone(), s["vc"].clone(), s["mass0"].clone()
    for b, n in enumerate(lengths(c)):
        if n <= c["budget"]:
            continue
        page, at = token_pages(s, c, b, n)
        for h in range(c["Hkv"]):
            # the positions are the slots here: the first `sink` and the last `recent` stay
            w = s["mass0"][page, h, at].double()
            w[:c["sink"]] = math.inf
            w[n - c["recent"]:] = math.inf
            kept = torch.argsort(-w, stable=True)[:c["budget"]]
            stays = torch.zeros(n, dtype=torch.bool, device=DEV)
            stays[kept] = True
            to = torch.nonzero(~stays[:c["budget"]])[:, 0]
            of = torch.nonzero(stays[c["budget"]:])[:, 0] + c["budget"]
            mass[page[to], h, at[to]] = mass[page[of], h, at[of]]
            for x in (k, v):
                y = x if c["layout"] == "HND" else x.transpose(1, 2)
                y[page[to], h, at[to]] = y[page[of], h, at[of]]
    return {"lens": None, "k": k.float(), "v": v.float(), "mass": mass, "positions": None}
