"""What the framework's operators for serving from an 8-bit paged cache are measured on: norms and
rotation of queries and keys, page tables built on the GPU, the append that fills the cache and the
read that takes its values out again, and the attention of new tokens over it.

``run`` computes an operator with elementary torch operations in 32 bits, angles in 64 (``own``
false), or calls the framework (``own`` true); ``exact`` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DEV = "cuda"
LEAST = 2.0 ** -100  # the least scale of a block


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the queries and keys of an 8K prompt of the grouped-head decoder, slices of one projection's output
        rope("rope_decoder8k", T=8192, Hq=32, Hkv=8, d=128, rot=128, dtype="bf16"),
        # one token of every sequence of a decode step, far into long contexts
        rope("rope_step", T=64, Hq=32, Hkv=8, d=128, rot=128, dtype="bf16", far=1 << 20),
        # a batch of odd length with neighbouring pairs, half of the channels rotated, heads before tokens
        rope("rope_partial", T=2 * 4097, B=2, Hq=16, Hkv=16, d=72, rot=36, dtype="fp16", layout="HND", pairs=True),
        # page tables of a decode step of many sequences, pages of 16 tokens
        assign("assign_step", B=256, lo=100, hi=4000, new_lo=1, new_hi=1, page=16, seed0=3),
        # page tables of new prompts, not all of which find pages
        assign("assign_prompts", B=48, lo=0, hi=0, new_lo=100, new_hi=4096, page=64, short=4, seed0=5),
        # a few ended sequences give their pages back, the others keep all
        release("release_ended", B=256, lo=100, hi=4000, keep="ended", page=16, seed0=7),
        # long prompts after an eviction down to 4096 tokens
        release("release_evicted", B=64, lo=6000, hi=32768, keep="cut", cut=4096, page=16, seed0=9),
        # one token of every sequence into the 8-bit cache, and the blocks they joined read back
        append("append_step", B=64, new=1, old=2007, Hkv=8, d=128, dtype="bf16", kt="int8", vt="e4m3", page=16, block=16),
        # the prompts of a batch into the cache, and read back in 16 bits as the next chunk's attention takes them
        append("append_prompts", B=16, new=4096, old=0, Hkv=8, d=128, dtype="bf16", kt="int8", vt="e4m3", page=64,
               block=64, layout="NHD", seed0=11),
        # one user, a short conversation: latency counts
        attn("attn_one", B=1, Hq=32, Hkv=8, lo=1000, hi=1000, d=128, dtype="bf16", kt="int8", vt="e4m3", page=16, block=16),
        # a serving batch of very different lengths, capped scores
        attn("attn_ragged32", B=32, Hq=32, Hkv=8, lo=128, hi=32768, d=128, dtype="bf16", kt="int8", vt="e4m3", page=64,
             block=64, layout="NHD", cap=50.0, seed0=13),
        # two long contexts, one key-value head per query head, biased by distance
        attn("attn_long", B=2, Hq=32, Hkv=32, lo=50001, hi=60001, d=64, dtype="fp16", kt="e4m3", vt="e4m3", page=128,
             block=32, bias=True, seed0=15),
    ]


def named(c, name, kw):
    return dict(c, **kw, **({"name": name} if name else {}))


def rope(name, **kw):
    return named(dict(op="rope", B=1, layout="packed", pairs=False, far=0), name, kw)


def assign(name, **kw):
    return named(dict(op="assign", short=0, seed0=0), name, kw)


def release(name, **kw):
    return named(dict(op="release", cut=0, seed0=0), name, kw)


def append(name, **kw):
    return named(dict(op="append", layout="HND", seed0=0), name, kw)


def attn(name, **kw):
    return named(dict(op="attn", layout="HND", cap=0.0, bias=False, seed0=0), name, kw)


def log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "assign", "release", "append", "append", "attn", "attn", "attn", "attn"])
    d = rng.choice([64, 64, 128, 128, 128, 32, 72, 80, 96, 120, 36])
    dtype, layout, seed = rng.choice(["fp16", "bf16"]), rng.choice(["HND", "NHD"]), rng.randrange(1 << 20)
    page = rng.choice([8, 16, 16, 32, 48, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    kt, vt = rng.choice(["int8", "e4m3"]), rng.choice(["int8", "e4m3"])
    block = rng.choice([b for b in (1, 4, 8, 16, 16, 24, 32, 64, 128) if page % b == 0])
    if op == "rope":
        hq = hkv * rng.choice([1, 2, 4, 7])
        b = rng.choice([1, 1, 2, 3])
        t = b * log_int(rng, 1, min(20000, 8192 * 40 * 128 // (b * (hq + hkv) * d)))
        return rope("", T=t, B=b, Hq=hq, Hkv=hkv, d=d, rot=rng.choice([d, d, d // 4 * 2]), dtype=dtype,
                    layout=rng.choice(["packed", layout]) if b == 1 else layout, pairs=rng.random() < 0.4,
                    far=rng.choice([0, 0, 1 << 20, 1 << 30]))
    if op == "assign":
        b = log_int(rng, 1, 1500)
        hi = rng.choice([0, 50, 4000])
        new = rng.choice([1, 1, 2, log_int(rng, 2, max(2, 100000 // b))])
        return assign("", B=b, lo=hi // 10, hi=hi, new_lo=max(1, new // 20), new_hi=new, page=page,
                      short=rng.choice([0, 0, 1, b // 3]), seed0=seed)
    if op == "release":
        b = log_int(rng, 1, 1500)
        hi = log_int(rng, 10, max(10, min(60000, 60000 * page // b)))
        return release("", B=b, lo=hi // rng.choice([1, 2, 10]), hi=hi, keep=rng.choice(["ended", "cut"]), cut=hi // 3,
                       page=page, seed0=seed)
    if op == "append":
        b = log_int(rng, 1, 64)
        new = rng.choice([1, log_int(rng, 1, max(1, 60000 // b))])
        return append("", B=b, new=new, old=rng.choice([0, 77, 1000]), Hkv=hkv, d=d, dtype=dtype, kt=kt, vt=vt, page=page,
                      block=block, layout=layout, seed0=seed)
    hi = log_int(rng, 20, 60000)
    b = log_int(rng, 1, 64)
    while b > 1 and b * hkv * hi * d > 32 * 8 * 20000 * 128:
        b -= 1
    return attn("", B=b, Hq=hkv * rng.choice([1, 2, 4, 8, 7, 16]), Hkv=hkv, lo=max(1, rng.choice([hi, hi // 2, hi // 50])),
                hi=hi, d=d, dtype=dtype, kt=kt, vt=vt, page=page, block=block, layout=layout,
                cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.3, seed0=seed)


# ------------------------------------------------------- what a case says apart from the values
def held(c):
    """Tokens that the sequences of a case hold before the call, the first one `hi`."""
    r = random.Random(c["seed0"])
    if c["op"] == "append":
        return [c["old"]] * c["B"]
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["B"] - 1)]


def added(c):
    """New tokens of each sequence."""
    r = random.Random(c["seed0"] + 1)
    if c["op"] == "append":
        return [c["new"]] + [r.randint(max(1, c["new"] // 4), c["new"]) for _ in range(c["B"] - 1)]
    return [c["new_hi"]] + [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"] - 1)]


def kept(c):
    """What a release leaves of each sequence: all of it or nothing, or at most `cut` tokens."""
    r = random.Random(c["seed0"] + 2)
    if c["keep"] == "cut":
        return [min(n, c["cut"]) for n in held(c)]
    return [n if r.random() < 0.9 else 0 for n in held(c)]


def pages_of(n, c):
    return -(-n // c["page"])


def work(c):
    if c["op"] == "rope":
        return {"bytes": 4 * c["T"] * (c["Hq"] + c["Hkv"]) * c["d"] + 4 * c["T"], "flops": 0}
    if c["op"] == "assign":
        taken = sum(pages_of(n + m, c) - pages_of(n, c) for n, m in zip(held(c), added(c)))
        return {"bytes": 12 * sum(added(c)) + 8 * taken + 20 * c["B"], "flops": 0}
    if c["op"] == "release":
        given = sum(pages_of(n, c) - pages_of(m, c) for n, m in zip(held(c), kept(c)))
        return {"bytes": 8 * given + 8 * c["B"], "flops": 0}
    if c["op"] == "append":
        # new rows in, codes out; codes in, values out of what is read back
        new, back = sum(added(c)), sum(read_back(c)[1])
        return {"bytes": 2 * c["Hkv"] * c["d"] * (3 * new + 3 * back), "flops": 0}
    n = sum(held(c))
    by = 2 * n * c["Hkv"] * (c["d"] + 4 / c["block"]) + 4 * c["B"] * c["Hq"] * c["d"] + 4 * c["B"] * c["Hq"]
    return {"bytes": by, "flops": 4 * n * c["Hq"] * c["d"]}


def read_back(c):
    """(first slots, counts) of the tokens that are read after an append: from the first block it touched on."""
    start = [n // c["block"] * c["block"] for n in held(c)]
    return start, [n + m - s for n, m, s in zip(held(c), added(c), start)]


# ------------------------------------------------------------------------------------ inputs
def normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def sums(v):
    cu = [0]
    for n in v:
        cu.append(cu[-1] + n)
    return cu


def slopes_of(heads):
    """A geometric row of slopes, as distance-biased attention uses."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32, device=DEV)


def needed(most, dtype):
    """The scale that a block of this largest magnitude needs."""
    if dtype == torch.int8:
        s = most / torch.full_like(most, 127.0)
    else:  # the smallest power of two with most <= 448 scale
        m, e = torch.frexp(most)  # most = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        s = torch.ldexp(torch.ones_like(most), torch.where(m > 0.875, e - 8, e - 9))
    return torch.clamp(s, min=LEAST)


def codes(x, dtype):
    return torch.clamp(torch.round(x), -127, 127).to(torch.int8) if dtype == torch.int8 else x.to(dtype)


def filled(g, shape, layout, block, dtype, offset):
    """A cache of normal values about a row of channel offsets, as codes and scales."""
    pages, hkv, page, d = shape
    x = torch.randn((pages, hkv, page // block, block, d), generator=g, device=DEV)
    if offset is not None:
        x += offset.view(1, hkv, 1, 1, d)
    s = needed(x.abs().amax((3, 4)), dtype)
    x *= (1.0 / s)[..., None, None]
    x = codes(x, dtype).view(shape)
    return (x if layout == "HND" else x.view(torch.uint8).transpose(1, 2).contiguous().view(dtype)), s


def tables(c, g, need):
    width, pages = max(need), sum(need) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table, at = torch.zeros((len(need), width), dtype=torch.int32, device=DEV), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order, at


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        prepare_rope(s, c, g)
        return s
    if c["op"] in ("assign", "release"):
        lens = held(c)
        grown = [n + m for n, m in zip(lens, added(c))] if c["op"] == "assign" else lens
        want, have = [pages_of(n, c) for n in grown], [pages_of(n, c) for n in lens]
        s["table"], order, _ = tables(c, g, want)
        # the first `have` pages of each sequence are held; the others are on the stack, in random order
        mask = torch.arange(s["table"].shape[1], device=DEV)[None] < ints(have)[:, None]
        taken = torch.zeros(order.numel(), dtype=torch.bool, device=DEV)
        taken[s["table"][mask].long()] = True
        free = order[~taken[order.long()]]
        s["table"] = torch.where(mask, s["table"], -1).contiguous()
        s["free"] = torch.zeros(order.numel(), dtype=torch.int32, device=DEV)
        s["free"][:free.numel()] = free
        count = free.numel()
        if c["op"] == "assign" and c["short"]:  # the last `short` sequences find no pages
            count = max(0, sum(want) - sum(have) - max(1, sum(want[-c["short"]:]) - sum(have[-c["short"]:])))
        s["count"], s["lens"] = ints([count]), ints(lens)
        if c["op"] == "assign":
            s["new"], s["tokens"] = ints(added(c)), sum(added(c))
        else:
            s["kept"] = ints(kept(c))
        return s
    dt, kt, vt, hnd = DTYPES[c["dtype"]], DTYPES[c["kt"]], DTYPES[c["vt"]], c["layout"] == "HND"
    lens = held(c)
    all_lens = [n + m for n, m in zip(lens, added(c))] if c["op"] == "append" else lens
    s["table"], order, _ = tables(c, g, [pages_of(n, c) for n in all_lens])
    shape = (order.numel(), c["Hkv"], c["page"], c["d"])
    offset = torch.randn((c["Hkv"], c["d"]), generator=g, device=DEV)
    s["kc"], s["ks"] = filled(g, shape, c["layout"], c["block"], kt, offset)
    s["vc"], s["vs"] = filled(g, shape, c["layout"], c["block"], vt, None)
    s["lens"] = ints(lens)
    if c["op"] == "attn":
        s["q"] = normal(g, (c["B"], c["Hq"], c["d"]), dt, 2.0)
        s["slopes"] = slopes_of(c["Hq"]) if c["bias"] else None
        return s
    t = sum(added(c))
    s["k"] = (torch.randn((t, c["Hkv"], c["d"]), generator=g, device=DEV) + offset).to(dt)
    s["v"] = normal(g, (t, c["Hkv"], c["d"]), dt)
    s["cu"], s["step"] = ints(sums(added(c))), c["new"] == 1
    s["seq"] = torch.repeat_interleave(torch.arange(c["B"], device=DEV), ints(added(c)).long())
    start, count = read_back(c)
    s["start"], s["count"], s["cu_back"], s["back"] = ints(start), ints(count), ints(sums(count)), sum(count)
    s["seq_back"] = torch.repeat_interleave(torch.arange(c["B"], device=DEV), s["count"].long())
    s["all_lens"] = ints(all_lens)
    return s


def prepare_rope(s, c, g):
    hq, hkv, d, b = c["Hq"], c["Hkv"], c["d"], c["B"]
    n, dt = c["T"] // b, DTYPES[c["dtype"]]
    # rows as a projection leaves them: queries, keys and values of a token side by side, uneven over the heads
    x = torch.randn((b, n, hq + 2 * hkv, d), generator=g, device=DEV)
    x = (x * torch.exp(torch.randn((hq + 2 * hkv, 1), generator=g, device=DEV))).to(dt)
    q, k = x[:, :, :hq], x[:, :, hq:hq + hkv]
    if c["layout"] == "packed":
        q, k = q[0], k[0]
    elif c["layout"] == "HND":
        q, k = q.transpose(1, 2), k.transpose(1, 2)
    s["q"], s["k"] = q, k
    s["wq"], s["wk"] = (normal(g, (d,), scale=0.2).add_(1.0).to(dt) for _ in "qk")
    first = torch.randint(0, c["far"] + 1, (b, 1), generator=g, device=DEV)
    pos = (first + torch.arange(n, device=DEV)).to(torch.int32)
    if c["far"] and n <= 256:  # a decode step: one token of each of many sequences
        pos = torch.randint(0, c["far"], (b, n), generator=g, device=DEV, dtype=torch.int32)
    s["pos"] = pos[0].contiguous() if c["layout"] == "packed" else pos
    s["freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])).float()


# ------------------------------------------------------------------------------------ passes
def run(s):
    return {"rope": run_rope, "assign": run_assign, "release": run_release, "append": run_append,
            "attn": run_attn}[s["case"]["op"]](s, s["case"])


def run_rope(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        layout = "NHD" if c["layout"] == "packed" else c["layout"]
        q, k = qa.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"], eps=1e-6, tensor_layout=layout,
                               interleaved=c["pairs"])
        return {"q": q, "k": k}
    angle = s["pos"].double()[..., None] * s["freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    heads = -3 if c["layout"] == "HND" else -2
    cos, sin = cos.unsqueeze(heads), sin.unsqueeze(heads)

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        r = c["rot"]
        if c["pairs"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((z, y[..., r:]), -1).to(x.dtype)
    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def run_assign(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        p = qa.paged_assign(s["table"], s["lens"], s["new"], s["free"], s["count"], c["page"], s["tokens"])
        return {"table": s["table"], "lens": p.seq_lens, "held": p.held_lens, "cu": p.cu_seqlens,
                "positions": p.positions, "slots": p.slots, "count": p.free_count}
    P, lens, new = c["page"], s["lens"].long(), s["new"].long()
    cu = torch.cat((torch.zeros_like(new[:1]), torch.cumsum(new, 0)))
    have, want = (lens + P - 1) // P, (lens + new + P - 1) // P
    need = want - have
    last = torch.cumsum(need, 0)
    served = (need == 0) | (last <= s["count"])
    j = torch.arange(s["table"].shape[1], device=DEV)[None]
    mine = (j >= have[:, None]) & (j < want[:, None]) & served[:, None]
    at = s["count"] - 1 - ((last - need)[:, None] + j - have[:, None])
    s["table"] = torch.where(mine, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"])
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = lens[b] + t - cu[b]
    slots = torch.where(served[b], s["table"][b, pos // P].long() * P + pos % P, -1)
    return {"table": s["table"], "lens": torch.where(served, lens + new, lens).int(),
            "held": torch.where(served, lens, -1).int(), "cu": cu.int(), "positions": pos.int(), "slots": slots,
            "count": (s["count"] - torch.where(served, need, 0).sum()).int()}


def run_release(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        count = qa.paged_release(s["table"], s["lens"], s["kept"], s["free"], s["count"], c["page"])
        return {"free": s["free"], "count": count}
    P, n = c["page"], s["free"].numel()
    have, keep = (s["lens"].long() + P - 1) // P, (s["kept"].long() + P - 1) // P
    given = have - keep
    first = s["count"] + torch.cumsum(given, 0) - given
    j = torch.arange(s["table"].shape[1], device=DEV)[None]
    mine = (j >= keep[:, None]) & (j < have[:, None])
    at = torch.where(mine, first[:, None] + j - keep[:, None], n)
    wide = torch.cat((s["free"], s["free"][:1]))
    s["free"].copy_(wide.scatter(0, at.flatten(), s["table"].flatten())[:n])
    return {"free": s["free"], "count": (s["count"] + given.sum()).int()}


def rows(cache, page, at, layout):
    """Rows of a cache as [tokens, heads, d] bytes."""
    x = cache.view(torch.uint8)
    return x[page, :, at] if layout == "HND" else x[page, at]


def set_rows(cache, page, at, layout, value):
    x = cache.view(torch.uint8)
    if layout == "HND":
        x[page, :, at] = value.view(torch.uint8)
    else:
        x[page, at] = value.view(torch.uint8)


def run_append(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        qa.paged_append_q8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"],
                           cu_seqlens=None if s["step"] else s["cu"], tensor_layout=c["layout"])
        k, v = qa.paged_read_q8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["all_lens"], s["cu_back"], s["back"],
                                starts=s["start"], dtype=s["k"].dtype, tensor_layout=c["layout"])
        return {"k": k, "v": v, "k_scales": s["ks"], "v_scales": s["vs"]}
    table, lens, P, G = s["table"].long(), s["lens"].long(), c["page"], c["block"]
    slot = torch.arange(s["seq"].numel(), device=DEV) - s["cu"].long()[s["seq"]] + lens[s["seq"]]
    page, at = table[s["seq"], slot // P], slot % P
    # the tokens that share their block with the first new ones
    old = (lens // G * G)[:, None] + torch.arange(G, device=DEV)
    joined = old < lens[:, None]
    old_page, old_at = table.gather(1, (old // P).clamp(max=table.shape[1] - 1)), old % P

    def store(x, cache, scales):
        dt, flat = cache.dtype, scales.transpose(1, 2).flatten(0, 1)  # [pages * blocks, heads], a copy
        x = x.float()
        block = page * (P // G) + at // G
        most = torch.zeros_like(flat).index_reduce_(0, block, x.abs().amax(-1), "amax")
        grown = needed(most, dt)
        # a block that starts with a new token has no scale yet
        begun = torch.ones(flat.shape[0], dtype=torch.bool, device=DEV)
        begun[(old_page * (P // G) + old_at // G)[joined]] = False
        grown = torch.where(begun[:, None], grown, torch.maximum(flat, grown))
        ob = old_page * (P // G) + old_at // G
        codes_old = rows(cache, old_page.flatten(), old_at.flatten(), c["layout"]).view(dt).float()
        again = codes(codes_old * (flat[ob.flatten()] / grown[ob.flatten()])[..., None], dt).view(torch.uint8)
        keep = joined.flatten()
        set_rows(cache, old_page.flatten()[keep], old_at.flatten()[keep], c["layout"], again[keep])
        set_rows(cache, page, at, c["layout"], codes(x * (1.0 / grown[block])[..., None], dt))
        touched = torch.zeros(flat.shape[0], dtype=torch.bool, device=DEV)
        touched[block] = True
        new = torch.where(touched[:, None], grown, flat)
        scales.copy_(new.view(scales.shape[0], P // G, -1).transpose(1, 2))

    store(s["k"], s["kc"], s["ks"])
    store(s["v"], s["vc"], s["vs"])
    t = torch.arange(s["back"], device=DEV) - s["cu_back"].long()[s["seq_back"]] + s["start"].long()[s["seq_back"]]
    page, at = table[s["seq_back"], t // P], t % P

    def read(cache, scales):
        x = rows(cache, page, at, c["layout"]).view(cache.dtype).float()
        return (x * scales[page, :, at // G][..., None]).to(s["k"].dtype)
    return {"k": read(s["kc"], s["ks"]), "v": read(s["vc"], s["vs"]), "k_scales": s["ks"], "v_scales": s["vs"]}


def run_attn(s, c):
    if own:
        import quantized_attention_mean_gb300 as qa
        out, lse = qa.paged_attn_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], c["hi"],
                                    tensor_layout=c["layout"], softcap=c["cap"], slopes=s["slopes"], return_lse=True)
        return {"out": out, "lse": lse}

    def gathered(cache, scales):
        x = cache.view(torch.uint8)[s["table"].long()].view(cache.dtype).float()
        x = x.transpose(1, 2) if c["layout"] == "HND" else x.permute(0, 3, 1, 2, 4)
        w = scales[s["table"].long()].transpose(1, 2).flatten(2, 3)
        return x.flatten(2, 3) * w.repeat_interleave(c["block"], 2)[..., None]
    k, v = gathered(s["kc"], s["ks"]), gathered(s["vc"], s["vs"])
    B, Hkv, L, d = k.shape
    g = c["Hq"] // Hkv
    t = torch.matmul(s["q"].float().view(B, Hkv, g, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if c["cap"]:
        t = c["cap"] * torch.tanh(t / c["cap"])
    j = torch.arange(L, device=DEV)
    if c["bias"]:
        t = t - s["slopes"].view(1, Hkv, g, 1) * (s["lens"][:, None] - 1 - j).abs().float().view(B, 1, 1, L)
    t = torch.where((j < s["lens"][:, None]).view(B, 1, 1, L), t, -math.inf)
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - m)
    total = p.sum(-1, keepdim=True)
    out = (torch.matmul(p, v) / total).view(B, c["Hq"], d).to(s["q"].dtype)
    return {"out": out, "lse": (m + torch.log(total)).view(B, c["Hq"])}


# ------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] in ("assign", "release"):
        return None
    s = prepare(case, seed)
    return {"rope": exact_rope, "append": exact_append, "attn": exact_attn}[case["op"]](s, s["case"])


def exact_rope(s, c):
    # one complex number per pair, turned by its angle
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[..., None] * s["freq"].double())
    turn = turn[..., None, :, :] if c["layout"] == "HND" else turn[..., None, :]

    def one(x, w):
        y = x.double()
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double()
        out, n = y.clone(), c["rot"] // 2
        first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if c["pairs"] else (slice(0, n), slice(n, 2 * n))
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        out[..., first], out[..., second] = z.real, z.imag
        return out
    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def token_rows(s, c, cache, b, lo, hi):
    """[tokens, heads, d] codes of slots lo.. of sequence b, in 64 bits."""
    slot = torch.arange(lo, hi, device=DEV)
    page, at = s["table"][b].long()[slot // c["page"]], slot % c["page"]
    x = cache.view(torch.uint8)
    x = x[page, :, at] if c["layout"] == "HND" else x[page, at]
    return x.view(cache.dtype).to(torch.float32).double()


def block_scales(s, c, scales, b, lo, hi):
    """[blocks, heads] scales of the blocks of slots lo.. (lo at a block's start), and where they lie."""
    first = torch.arange(lo, hi, c["block"], device=DEV)
    page, at = s["table"][b].long()[first // c["page"]], first % c["page"] // c["block"]
    return scales[page, :, at].double(), page, at


def exact_append(s, c):
    G, cu = c["block"], sums(added(c))
    start, count = read_back(c)
    out, planes = {}, {}
    for name, x, cache, scales in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        parts, plane = [], scales.double()
        for b, (n, m) in enumerate(zip(held(c), added(c))):
            lo, hi = start[b], n + m
            fresh = x[cu[b]:cu[b + 1]].double()
            pad = -(hi - lo) % G
            held_rows = token_rows(s, c, cache, b, lo, n)
            was, page, at = block_scales(s, c, scales, b, lo, hi)
            most = torch.cat((torch.zeros_like(held_rows), fresh, fresh.new_zeros((pad, *fresh.shape[1:]))))
            most = most.abs().amax(-1).view(-1, G, fresh.shape[1]).amax(1)
            if cache.dtype == torch.int8:
                scale = most / 127
            else:
                scale = torch.exp2(torch.ceil(torch.log2(torch.clamp(most, min=1e-300) / 448)))
            scale = torch.clamp(scale, min=LEAST)
            if n > lo:
                scale[0] = torch.maximum(scale[0], was[0])
            plane[page, :, at] = scale
            each = scale.repeat_interleave(G, 0)[:hi - lo, :, None]
            units = torch.cat((held_rows * was[0][None, :, None], fresh)) / each
            if cache.dtype == torch.int8:
                units = torch.round(units)
            else:  # three bits behind the leading one, steps of 2^-9 at the bottom
                step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(units.abs(), min=1e-300))), min=-6.0) - 3)
                units = torch.round(units / step) * step
            parts.append(units * each)
        out[name], planes[name] = torch.cat(parts), plane
    return {"k": out["k"], "v": out["v"], "k_scales": planes["k"], "v_scales": planes["v"]}


def exact_attn(s, c):
    g = c["Hq"] // c["Hkv"]
    out = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((c["B"], c["Hq"]), dtype=torch.float64, device=DEV)
    for b, n in enumerate(held(c)):
        k, v = (token_rows(s, c, cache, b, 0, n) * block_scales(s, c, w, b, 0, n)[0].repeat_interleave(c["block"], 0)[:n, :, None]
                for cache, w in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        q = s["q"][b].double().view(c["Hkv"], g, c["d"])
        t = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(c["d"])
        if c["cap"]:
            t = torch.tanh(t / c["cap"]) * c["cap"]
        if c["bias"]:
            t = t - s["slopes"].double().view(c["Hkv"], g, 1) * torch.arange(n - 1, -1, -1, device=DEV)
        lse[b] = torch.logsumexp(t, -1).flatten()
        out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(t, -1), v).reshape(c["Hq"], c["d"])
    return {"out": out, "lse": lse}
