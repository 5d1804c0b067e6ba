"""Page tables on the GPU against plain loops: every result is a whole number and has to be equal."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def pages_of(n, size):
    return -(-n // size)


def assign(table, lens, add, free, count, size, most, base=None):
    """The definition, sequence by sequence, on lists."""
    cap = len(free)
    top = max(0, min(count, cap))
    room, width = len(table[0]) * size if table else 0, 0
    new, held, cu, pos, slots, tokens, stuck, low = [], [], [0], [-1] * most, [-1] * most, 0, False, top
    wanted = 0
    for b, (n, m) in enumerate(zip(lens, add)):
        bad = n < 0 or m < 0 or n + m > room
        begin, end = tokens, tokens + max(m, 0)
        tokens = end
        need = 0 if bad else pages_of(n + m, size) - pages_of(n, size)
        wanted += need
        ok = not bad and end <= most and (need == 0 or wanted <= top)
        if ok and need:
            first = top - 1 - (wanted - need)
            for i in range(need):
                table[b][pages_of(n, size) + i] = free[first - i]
            low = top - wanted
        new.append(n + m if ok else n)
        held.append(n if ok else -1)
        cu.append(min(end, most))
        for t in range(min(begin, most), min(end, most)):
            at = n + t - begin
            pos[t] = (n if base is None else base[b]) + t - begin
            if ok:
                pg = table[b][at // size]
                if 0 <= pg < cap:
                    slots[t] = pg * size + at % size
    return new, held, cu, pos, slots, low


CASES = [
    # lens, new tokens, page size, width, pages on the stack, room for tokens
    ([0], [1], 16, 2, 4, 1),
    ([0, 5, 16, 31], [17, 1, 1, 1], 16, 3, 20, 20),
    ([0, 0, 0, 0], [100, 64, 63, 65], 64, 2, 4, 292),                 # the third finds no page, nor does the fourth
    ([10, 3, 7], [0, 0, 0], 4, 4, 0, 0),                              # nothing to do
    ([3, 60, 0], [1, 10, 4], 4, 16, 3, 30),                           # no room in the second's row
    ([-1, 5, 4], [3, -2, 2], 4, 8, 9, 12),                            # bad lengths
    ([0, 0, 0], [5, 5, 5], 4, 4, 12, 12),                             # the last one's tokens end behind the maps
    ([i % 37 for i in range(1000)], [1] * 1000, 8, 8, 400, 1000),     # runs out halfway
    ([0] * 3, [5000, 1, 9000], 16, 600, 900, 14100),
    ([100000], [30000], 128, 1100, 300, 30000),
    ([i % 5 for i in range(70000 // 4)], [i % 4 for i in range(70000 // 4)], 2, 8, 100000, 30000),
]


@pytest.mark.parametrize("lens,add,size,width,stack,most", CASES)
@pytest.mark.parametrize("based", [False, True])
def test_assign(lens, add, size, width, stack, most, based):
    import quantized_attention_mean_gb300 as qa
    B = len(lens)
    g = torch.Generator().manual_seed(B + stack)
    pages = stack + sum(pages_of(max(n, 0), size) for n in lens)
    order = torch.randperm(pages, generator=g).tolist()
    table = [[-9] * width for _ in lens]
    at = stack
    for b, n in enumerate(lens):
        for i in range(min(width, pages_of(max(n, 0), size))):
            table[b][i] = order[at]
            at += 1
    free = order[:stack] + [-5] * (pages - stack)
    base = [1000 * b + 7 for b in range(B)] if based else None
    wide = torch.full((B, width + 3), -77, dtype=torch.int32, device=DEV)
    wide[:, :width] = ints(table)
    ws = qa.alloc_workspace(256, DEV).fill_(255)
    a = qa.paged_assign(wide[:, :width], ints(lens), ints(add), ints(free), ints([stack]), size, most,
                        next_positions=None if base is None else ints(base), workspace=ws)
    want = assign(table, lens, add, free, stack, size, most, base)
    assert a.seq_lens.tolist() == want[0] and a.held_lens.tolist() == want[1] and a.cu_seqlens.tolist() == want[2]
    assert a.positions.tolist() == want[3] and a.slots.tolist() == want[4] and a.free_count.tolist() == [want[5]]
    assert wide[:, :width].tolist() == table and (wide[:, width:] == -77).all()
    bad = any(n < 0 or m < 0 or n + m > width * size for n, m in zip(lens, add)) or sum(max(m, 0) for m in add) > most
    assert qa.read_device_status(ws) == (12 if bad else 0)


def test_assign_counts_and_pages_out_of_range():
    import quantized_attention_mean_gb300 as qa
    ws = qa.alloc_workspace(256, DEV)
    for said, top in ((99, 3), (-4, 0)):
        table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
        a = qa.paged_assign(table, ints([0, 0]), ints([3, 3]), ints([4, 5, 6]), ints([said]), 4, 6, workspace=ws)
        assert qa.read_device_status(ws) == 12
        assert a.free_count.item() == (1 if top else 0) and a.held_lens.tolist() == ([0, 0] if top else [-1, -1])
    # a held page outside of the cache: its token has no slot
    table = ints([[50, -1], [1, -1]])
    a = qa.paged_assign(table, ints([2, 2]), ints([1, 1]), ints([0, 1, 2]), ints([1]), 4, 2, workspace=ws)
    assert qa.read_device_status(ws) == 13 and a.slots.tolist() == [-1, 6]
    # no sequences at all, and no pages at all
    none = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    a = qa.paged_assign(none, ints([]), ints([]), ints([1, 2]), ints([2]), 4, 3)
    assert a.cu_seqlens.tolist() == [0] and a.free_count.item() == 2 and a.slots.tolist() == [-1] * 3
    a = qa.paged_assign(torch.zeros(1, 0, dtype=torch.int32, device=DEV), ints([0]), ints([1]), ints([]), ints([0]), 4, 1)
    assert a.held_lens.tolist() == [-1] and a.free_count.item() == 0


def release(table, lens, keep, free, count, size):
    cap, top = len(free), max(0, min(count, len(free)))
    high, sum_ = top, 0
    for b, (n, m) in enumerate(zip(lens, keep)):
        if m < 0 or m > n or n > len(table[b]) * size:
            continue
        given = table[b][pages_of(m, size):pages_of(n, size)]
        if any(not 0 <= p < cap for p in given):
            continue
        sum_ += len(given)
        if given and top + sum_ <= cap:
            free[top + sum_ - len(given):top + sum_] = given
            high = top + sum_
    return high


@pytest.mark.parametrize("lens,keep,size,count,bad", [
    ([5], [0], 4, 0, False),
    ([5, 8, 9, 0], [5, 7, 4, 0], 4, 3, False),
    ([40, 41, 3], [-1, 50, 0], 4, 2, True),                           # lengths out of range give nothing
    ([i % 97 for i in range(700)], [(i % 97) // 2 for i in range(700)], 8, 50, False),
    ([20000, 1, 30000], [4096, 0, 29999], 16, 10, False),
    ([1000] * 20000, [0] * 20000, 1000, 0, False),
])
def test_release(lens, keep, size, count, bad):
    import quantized_attention_mean_gb300 as qa
    width = max(pages_of(n, size) for n in lens)
    pages = sum(pages_of(n, size) for n in lens) + count
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(len(lens))).tolist()
    table, at = [], count
    for n in lens:
        k = pages_of(n, size)
        table.append(order[at:at + k] + [-3] * (width - k))
        at += k
    free = order[:count] + [-1] * (pages - count)
    stack, ws = ints(free), qa.alloc_workspace(qa.paged_release_workspace_bytes(len(lens)), DEV).fill_(255)
    new = qa.paged_release(ints(table), ints(lens), ints(keep), stack, ints([count]), size, workspace=ws)
    high = release(table, lens, keep, free, count, size)
    assert new.tolist() == [high] and stack.tolist() == free
    assert qa.read_device_status(ws) == (12 if bad else 0)
    again = ints(order[:count] + [-1] * (pages - count))
    assert qa.paged_release(ints(table), ints(lens), ints(keep), again, ints([count]), size).tolist() == [high]
    assert torch.equal(again, stack)


def test_release_of_bad_pages_and_without_room():
    import quantized_attention_mean_gb300 as qa
    ws = qa.alloc_workspace(qa.paged_release_workspace_bytes(3), DEV)
    table = [[0, 1], [2, 9], [3, 4]]
    stack = ints([5, -1, -1, -1, -1, -1])
    new = qa.paged_release(ints(table), ints([8, 8, 8]), ints([0, 0, 0]), stack, ints([1]), 4, workspace=ws)
    assert qa.read_device_status(ws) == 13
    assert new.item() == 5 and stack.tolist() == [5, 0, 1, 3, 4, -1]
    stack = ints([5, -1, -1, -1])
    table[1] = [2, 3]
    new = qa.paged_release(ints(table), ints([8, 8, 4]), ints([0, 0, 0]), stack, ints([1]), 4, workspace=ws)
    assert qa.read_device_status(ws) == 12                             # (the third would fit, but the second does not)
    assert new.item() == 3 and stack.tolist() == [5, 0, 1, -1]
    none = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    assert qa.paged_release(none, ints([]), ints([]), stack, ints([2]), 4).item() == 2


@pytest.mark.parametrize("said,count,status", [(2, 2, 0), (9, 4, 12), (-3, 0, 12)])
def test_no_sequences_and_a_count_out_of_range(said, count, status):
    # with no sequence the count is clamped and told of as with some
    import quantized_attention_mean_gb300 as qa
    none, free = torch.zeros(0, 3, dtype=torch.int32, device=DEV), ints([7, 8, 9, 10])
    ws = qa.alloc_workspace(qa.paged_release_workspace_bytes(0), DEV).fill_(255)
    a = qa.paged_assign(none, ints([]), ints([]), free, ints([said]), 4, 2, workspace=ws)
    assert qa.read_device_status(ws) == status
    assert a.free_count.item() == count and a.cu_seqlens.tolist() == [0] and a.positions.tolist() == [-1, -1]
    ws.fill_(255)
    assert qa.paged_release(none, ints([]), ints([]), free, ints([said]), 4, workspace=ws).item() == count
    assert qa.read_device_status(ws) == status
    assert qa.paged_release(none, ints([]), ints([]), free, ints([said]), 4).item() == count
    assert free.tolist() == [7, 8, 9, 10]


def test_pages_go_round():
    # random growth and ends over many steps: no page is ever held twice, and none is lost
    import quantized_attention_mean_gb300 as qa
    g = torch.Generator().manual_seed(6)
    B, size, width, pages = 37, 4, 12, 160
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free, count = torch.arange(pages, dtype=torch.int32, device=DEV), ints([pages])
    lens = ints([0] * B)
    for _ in range(30):
        add = torch.randint(0, 9, (B,), generator=g, dtype=torch.int32).to(DEV)
        add = torch.minimum(add, width * size - lens)
        a = qa.paged_assign(table, lens, add, free, count, size, 8 * B)
        lens, count = a.seq_lens, a.free_count
        keep = torch.where(torch.rand(B, generator=g).to(DEV) < 0.2, lens // 3, lens)
        count = qa.paged_release(table, lens, keep, free, count, size)
        lens = keep
        held = [p for row, n in zip(table.tolist(), lens.tolist()) for p in row[:pages_of(n, size)]]
        assert sorted(held + free[:count.item()].tolist()) == list(range(pages))
