"""A paged cache on the CPU, and append and eviction on it by plain loops."""

import math

import torch


def make_cache(lens, hkv, d, page_size, dtype=torch.bfloat16, layout="HND", spare=3, seed=0, room=0):
    """Random pages in random order; `room` more slots per sequence than it holds."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(n + room) // page_size) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32)  # unused entries: never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, hkv, page_size, d) if layout == "HND" else (pages, page_size, hkv, d)
    k, v = (torch.randn(shape, generator=g).to(dtype) for _ in "kv")
    return dict(k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32), layout=layout, size=page_size)


def place(c, b, n):
    """(pages, slots in them) of the first n token slots of sequence b."""
    t = torch.arange(n)
    return c["table"][b, t // c["size"]].long(), t % c["size"]


def rows(c, which, b, h, n):
    p, s = place(c, b, n)
    x = c[which]
    return x[p, h, s] if c["layout"] == "HND" else x[p, s, h]


def set_row(c, which, page, h, slot, value):
    if c["layout"] == "HND":
        c[which][page, h, slot] = value
    else:
        c[which][page, slot, h] = value


def get_row(c, which, page, h, slot):
    return (c[which][page, h, slot] if c["layout"] == "HND" else c[which][page, slot, h]).clone()


def evict(c, mass, pos, budget, sink, recent):
    """In place on c, mass and pos; returns the new lengths."""
    hkv = mass.shape[1]
    new = []
    for b, n in enumerate(c["lens"].tolist()):
        new.append(min(n, budget))
        if n <= budget:
            continue
        p, s = place(c, b, n)
        for h in range(hkv):
            w, q = mass[p, h, s].tolist(), pos[p, h, s].tolist()
            last = max(q)
            def key(j):
                if q[j] < sink or q[j] > last - recent:
                    return (1, 0.0)
                return (0, -math.inf if math.isnan(w[j]) else w[j])
            order = sorted(range(n), key=lambda j: (-key(j)[0], -key(j)[1], j))
            kept = set(order[:budget])
            to = [j for j in range(budget) if j not in kept]
            of = [j for j in range(budget, n) if j in kept]
            assert len(to) == len(of)
            for x, y in zip(to, of):
                for which in "kv":
                    set_row(c, which, p[x], h, s[x], get_row(c, which, p[y], h, s[y]))
                mass[p[x], h, s[x]] = mass[p[y], h, s[y]]
                pos[p[x], h, s[x]] = pos[p[y], h, s[y]]
    return torch.tensor(new, dtype=torch.int32)
