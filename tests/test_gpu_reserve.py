"""Page reservation against a stack of Python integers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rkv():
    from two_stage_kv_snapkv_gb300 import rkv as mod
    return mod


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """The definition: stack, tables and counts as lists."""

    def __init__(self, stack, tables, P, max_pages):
        self.stack, self.tables, self.P, self.max_pages = list(stack), [list(t) for t in tables], P, max_pages

    def reserve(self, lens, start):
        ok = [0 <= x <= self.max_pages * self.P for x in lens]
        need = [-(-x // self.P) if o else len(t) for x, o, t in zip(lens, ok, self.tables)]
        for b, t in enumerate(self.tables):
            while_kept, given = t[:need[b]], t[need[b]:]
            self.stack += given
            self.tables[b] = while_kept
        have, asked = len(self.stack), 0
        for b, t in enumerate(self.tables):
            take = need[b] - len(t)
            if take <= 0:
                continue
            asked += take
            if asked > have:
                ok[b] = False
                continue
            for _ in range(take):
                t.append(self.stack.pop())
        slots, first = [], [0]
        for b, t in enumerate(self.tables):
            if ok[b] and start[b] >= 0:
                slots += [t[x // self.P] * self.P + x % self.P for x in range(start[b], lens[b])]
            first.append(len(slots))
        return slots, first


def _check(pool, table, model):
    held = pool.held.cpu().tolist()
    assert held == [len(t) for t in model.tables]
    tab = table.cpu().tolist()
    for b, t in enumerate(model.tables):
        assert tab[b][:len(t)] == t, b
    count = int(pool.free_count)
    assert count == len(model.stack)
    assert pool.free_pages[:count].cpu().tolist() == model.stack
    assert int(pool.sync) == 0


@pytest.mark.parametrize("B,P,pages,phys", [(1, 16, 8, 3), (3, 32, 16, 40), (33, 64, 64, 900), (256, 16, 24, 5000)])
def test_sequences_grow_shrink_and_run_dry(rkv, B, P, pages, phys):
    g = torch.Generator().manual_seed(B)
    order = torch.randperm(phys, generator=g).to(torch.int32)
    pool = rkv.PagePool(phys, B, "cuda", free_pages=order.cuda())
    table = torch.full((B, pages), -7, dtype=torch.int32, device="cuda")
    model = Model(order.tolist(), [[] for _ in range(B)], P, pages)
    was = [0] * B
    dry = 0
    for step in range(12):
        lens = torch.randint(0, pages * P + 1, (B,), generator=g).tolist()
        if step % 3 == 1:
            lens = [min(x + 1, pages * P) for x in was]   # one more token each
        if step == 5:
            lens = [0] * B
        if step == 7:
            lens[0] = pages * P + 1                        # longer than its table
        start = [w if torch.rand(1, generator=g) < 0.8 else 0 for w in was]
        size = sum(max(0, x - s) for x, s in zip(lens, start)) + 5
        slots = torch.full((size,), -9, dtype=torch.int32, device="cuda")
        first = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        rkv.rkv_reserve_pages(pool, table, P, _ints(lens), start=_ints(start), slots=slots, first=first)
        ref, cu = model.reserve(lens, start)
        _check(pool, table, model)
        assert first.cpu().tolist() == cu
        assert slots.cpu().tolist() == ref + [-9] * (size - len(ref))
        unserved = any(0 <= x <= pages * P and -(-x // P) != len(t) for x, t in zip(lens, model.tables))
        want = (0x20 if unserved else 0) | (0x2 if step == 7 else 0)
        assert rkv.rkv_read_device_error(pool.error_word)[1] == want, step
        dry += unserved
        was = [min(x, len(t) * P) if 0 <= x <= pages * P else len(t) * P for x, t in zip(lens, model.tables)]
    if phys < B * pages // 2:  # less than the lengths ask for on average
        assert dry > 0


def test_counts_beside_the_old_ones(rkv):
    pool = rkv.PagePool(40, 2, "cuda")
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    held, count = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        rkv.rkv_reserve_pages(pool, table, 16, _ints([17, 64]), held_out=held, free_count_out=count)
        assert pool.held.tolist() == [0, 0] and int(pool.free_count) == 40
        assert held.tolist() == [2, 4] and int(count) == 34
        assert table[0, :2].tolist() == [0, 1] and table[1, :4].tolist() == [2, 3, 4, 5]
        assert table[0, 2:].tolist() == [-1] * 6


def test_counts_that_cannot_be(rkv):
    for held, count, bits in (([9, 1], 10, 0x20), ([-1, 1], 10, 0x20), ([0, 1], -1, 0x20), ([0, 1], 41, 0x20)):
        pool = rkv.PagePool(40, 2, "cuda", free_count=_ints([count]), held=_ints(held))
        table = torch.full((2, 8), 5, dtype=torch.int32, device="cuda")
        slots, first = torch.full((64,), -9, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
        rkv.rkv_reserve_pages(pool, table, 16, _ints([16, 32]), start=_ints([0, 30]), slots=slots, first=first)
        assert rkv.rkv_read_device_error(pool.error_word)[1] == bits
        if 0 <= count <= 40:  # the sequence whose count is sound is served
            assert pool.held.tolist() == [held[0], 2] and int(pool.free_count) == count - 1
            assert first.tolist() == [0, 0, 2]
        else:
            assert pool.held.tolist() == held and int(pool.free_count) == count
            assert first.tolist() == [0, 0, 0] and (slots == -9).all()


def test_slots_that_do_not_fit_and_bad_ids(rkv):
    pool = rkv.PagePool(4, 1, "cuda", free_pages=_ints([0, 99, -3, 2]))
    table = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    slots, first = torch.full((40,), -9, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    rkv.rkv_reserve_pages(pool, table, 16, _ints([60]), start=_ints([10]), slots=slots[:40], first=first)
    assert rkv.rkv_read_device_error(pool.error_word)[1] == 0x1 | 0x2
    assert first.tolist() == [0, 50]
    want = [2 * 16 + x for x in range(10, 16)] + [-1] * 32 + [0, 1]
    assert slots.tolist() == want
    rkv.rkv_reserve_pages(pool, table, 16, _ints([60]), start=_ints([-1]), slots=slots, first=first)
    assert rkv.rkv_read_device_error(pool.error_word)[1] == 0x2 and first.tolist() == [0, 0]
    assert rkv.rkv_read_device_error(pool.error_word) == (rkv.RKV_OK, 0)


def test_captured_step_follows_the_lengths(rkv):
    pool = rkv.PagePool(100, 4, "cuda")
    table = torch.full((4, 16), -1, dtype=torch.int32, device="cuda")
    lens, start = _ints([0, 5, 16, 31]), _ints([0, 0, 0, 0])
    slots, first = torch.full((4,), -9, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    rkv.rkv_reserve_pages(pool, table, 16, lens)
    model = Model(range(99, -1, -1), [[] for _ in range(4)], 16, 16)
    model.reserve([0, 5, 16, 31], [0] * 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        start.copy_(lens)
        lens += 1
        rkv.rkv_reserve_pages(pool, table, 16, lens, start=start, slots=slots, first=first)
    now = [0, 5, 16, 31]
    for _ in range(40):
        graph.replay()
        ref, _ = model.reserve([x + 1 for x in now], now)
        now = [x + 1 for x in now]
        torch.cuda.synchronize()
        _check(pool, table, model)
        assert slots.tolist() == ref


def test_slots_feed_the_bf16_cache(rkv):
    """Rows written through the slots are the rows that the append finds in place."""
    B, H, P, n = 3, 2, 16, [20, 1, 47]
    pool = rkv.PagePool(3 * 8 + 2, B, "cuda")
    table = torch.zeros(B, 8, dtype=torch.int32, device="cuda")
    slots, first = torch.empty(sum(n), dtype=torch.int32, device="cuda"), torch.empty(B + 1, dtype=torch.int32, device="cuda")
    rkv.rkv_reserve_pages(pool, table, P, _ints(n), start=_ints([0] * B), slots=slots, first=first)
    cache = rkv.PagedCache(B, H, P, 8, "cuda", page_table=table, num_phys_pages=26)
    g = torch.Generator(device="cuda").manual_seed(3)
    for b in range(B):
        k, v = (torch.randn(H, n[b], 128, generator=g, device="cuda").bfloat16() for _ in range(2))
        at = slots[int(first[b]):int(first[b + 1])].long()
        cache.k_pages[at // P, :, at % P] = k.transpose(0, 1)
        cache.v_pages[at // P, :, at % P] = v.transpose(0, 1)
        got_k, got_v = cache.token_kv(b, n[b])
        assert torch.equal(got_k, k) and torch.equal(got_v, v)
