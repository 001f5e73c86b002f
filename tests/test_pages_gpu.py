"""Pages of a pool (pa_pages_fork, pa_pages_resize, pa_pages_compact) against a
plain simulation, exactly: tables, lengths, counts and every byte of the caches."""
import random

import pytest
import torch

from decode_attention_paged_pa_gb300 import binding

pytestmark = pytest.mark.gpu


class Pool:
    """The operators' definition, one row and one block at a time (CPU)."""

    def __init__(self, seed, lens, MB, NB, BS, caches=((48,), (3, 32)), share=0):
        r = random.Random(seed)
        g = torch.Generator().manual_seed(seed)
        self.BS, self.MB, self.NB = BS, MB, NB
        ids = list(range(NB))
        r.shuffle(ids)
        self.tables = torch.randint(-9, 2 * NB, (len(lens), MB), generator=g, dtype=torch.int32)
        self.lens = list(lens)
        self.refs = [0] * NB
        for s, L in enumerate(lens):
            for j in range(-(-L // BS)):
                shared = s > 0 and j < share and j < lens[0] // BS
                self.tables[s, j] = int(self.tables[0, j]) if shared else ids.pop()
                self.refs[int(self.tables[s, j])] += 1
        self.caches = [torch.randint(0, 256, (NB,) + c, generator=g, dtype=torch.uint8).repeat_interleave(16, -1)
                       for c in caches]

    def copy(self, src, dst):
        for c in self.caches:
            c[dst] = c[src].clone()

    def free(self):
        return [b for b in range(self.NB) if self.refs[b] <= 0]

    def blocks(self, L):
        return -(-L // self.BS)

    def fork(self, parents, out, lens_out):
        free = self.free()
        if sum(1 for p in parents if p >= 0 and self.lens[p] % self.BS) > len(free):
            return False
        for i, p in enumerate(parents):
            L = self.lens[p] if p >= 0 else 0
            lens_out[i] = L
            for j in range(L // self.BS):
                out[i, j] = self.tables[p, j]
                self.refs[int(out[i, j])] += 1
            if L % self.BS:
                j, b = L // self.BS, free.pop(0)
                self.copy(int(self.tables[p, j]), b)
                out[i, j], self.refs[b] = b, 1
        return True

    def resize(self, new):
        free, before, old = self.free(), list(self.refs), self.tables.clone()
        plan = []
        for s, (L, N) in enumerate(zip(self.lens, new)):
            keep, a, b = min(L, N), self.blocks(L), self.blocks(N)
            cow = keep % self.BS != 0 and before[int(old[s, keep // self.BS])] > 1
            plan.append((L, N, keep, a, b, cow))
        if sum(p[5] + max(0, p[4] - p[3]) for p in plan) > len(free):
            return False
        for s, (L, N, keep, a, b, cow) in enumerate(plan):
            if cow:
                j, d = keep // self.BS, free.pop(0)
                self.copy(int(old[s, j]), d)
                self.refs[int(old[s, j])] -= 1
                self.tables[s, j], self.refs[d] = d, 1
            for j in range(a, b):
                d = free.pop(0)
                self.tables[s, j], self.refs[d] = d, 1
            for j in range(b, a):
                self.refs[int(old[s, j])] -= 1
            self.lens[s] = N
        return True

    def compact(self):
        used = [b for b in range(self.NB) if self.refs[b] > 0]
        holes = [b for b in range(len(used)) if self.refs[b] <= 0]
        movers = [b for b in used if b >= len(used)]
        new = {b: b for b in used}
        for s, d in zip(movers, holes):
            self.copy(s, d)
            self.refs[d], self.refs[s] = self.refs[s], 0
            new[s] = d
        for s, L in enumerate(self.lens):
            for j in range(self.blocks(L)):
                self.tables[s, j] = new[int(self.tables[s, j])]
        return [new.get(b, -1) for b in range(self.NB)]

    def on_gpu(self):
        dev = torch.device("cuda")
        return (self.tables.to(dev), i32(self.lens), i32(self.refs), [c.to(dev) for c in self.caches])

    def equals(self, tables, lens, refs, caches):
        assert torch.equal(tables.cpu(), self.tables)
        assert lens.tolist() == self.lens and refs.tolist() == self.refs
        for a, b in zip(caches, self.caches):
            assert torch.equal(a.cpu(), b)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def status(ws, want=binding.PA_OK):
    assert binding.device_status(ws) == want


SIZES = [  # (sequences, MB, blocks, block size)
    (1, 1, 3, 16), (7, 9, 100, 8), (40, 300, 4000, 1), (1100, 6, 9000, 16), (5, 5, 300001, 4),
]


@pytest.mark.parametrize("S,MB,NB,BS", SIZES)
def test_fork(S, MB, NB, BS):
    r = random.Random(S)
    lens = [r.choice([0, 1, BS, r.randint(0, min(MB * BS, NB // S * BS // 2))]) for _ in range(S)]
    p = Pool(S, lens, MB, NB, BS, share=2)
    n = min(2 * S + 1, sum(x == 0 for x in p.refs))
    parents = [r.randrange(-1, S) for _ in range(n)]
    tables, ld, refs, caches = p.on_gpu()
    out = torch.full((n, MB), -5, dtype=torch.int32, device="cuda")
    lo = i32([9] * n)
    ws = binding.pa_pages_fork(out, lo, tables, ld, i32(parents), refs, caches, BS)
    status(ws)
    want, wl = torch.full((n, MB), -5, dtype=torch.int32), [9] * n
    assert p.fork(parents, want, wl)
    p.equals(tables, ld, refs, caches)
    assert torch.equal(out.cpu(), want) and lo.tolist() == wl


@pytest.mark.parametrize("S,MB,NB,BS", SIZES)
def test_resize(S, MB, NB, BS):
    r = random.Random(S + 1)
    top = min(MB * BS, NB // S * BS // 2)
    lens = [r.choice([0, 1, BS, r.randint(0, top), r.randint(0, top)]) for _ in range(S)]
    p = Pool(S, lens, MB, NB, BS, share=3)
    tables, ld, refs, caches = p.on_gpu()
    for step in range(4):
        new = [r.choice([L, 0, max(0, L - 1), min(L + 1, top), r.randint(0, top)]) for L in p.lens]
        ws = binding.pa_pages_resize(tables, ld, i32(new), refs, caches, BS)
        status(ws)
        assert p.resize(new)
        p.equals(tables, ld, refs, caches)


@pytest.mark.parametrize("S,MB,NB,BS", SIZES)
def test_compact(S, MB, NB, BS):
    r = random.Random(S + 2)
    top = min(MB * BS, NB // S * BS // 2)
    p = Pool(S + 50, [r.randint(0, top) for _ in range(S)], MB, NB, BS, share=2)
    tables, ld, refs, caches = p.on_gpu()
    for step in range(2):  # the second time nothing is left to move
        ids = i32([7] * NB)
        ws = binding.pa_pages_compact(tables, ld, refs, caches, BS, new_ids=ids)
        status(ws)
        assert ids.tolist() == p.compact()
        p.equals(tables, ld, refs, caches)
    used = sum(x > 0 for x in p.refs)
    assert all(x > 0 for x in p.refs[:used])


def test_truncation_into_shared_blocks_copies_them():
    """Two rows cut back into the same shared block each get a copy; the third keeps it."""
    p = Pool(3, [40, 40, 40], 4, 20, 16, share=2)
    tables, ld, refs, caches = p.on_gpu()
    shared = int(p.tables[0, 1])
    ws = binding.pa_pages_resize(tables, ld, i32([20, 25, 40]), refs, caches, 16)
    status(ws)
    assert p.resize([20, 25, 40])
    p.equals(tables, ld, refs, caches)
    assert refs[shared] == 1 and int(tables[2, 1]) == shared


def test_too_few_blocks_changes_nothing():
    p = Pool(4, [30, 33], 8, 6, 16)
    tables, ld, refs, caches = p.on_gpu()
    ws = binding.pa_pages_resize(tables, ld, i32([100, 0]), refs, caches, 16)
    status(ws, binding.PA_ERR_NO_BLOCKS)
    p.equals(tables, ld, refs, caches)
    out, lo = torch.full((3, 8), -5, dtype=torch.int32, device="cuda"), i32([9, 9, 9])
    ws = binding.pa_pages_fork(out, lo, tables, ld, i32([0, 1, 0]), refs, caches, 16, workspace=ws.new_empty(4096))
    status(ws, binding.PA_ERR_NO_BLOCKS)
    p.equals(tables, ld, refs, caches)
    assert bool((out == -5).all()) and lo.tolist() == [9, 9, 9]
    # Blocks given back are free for the next call.
    ws = binding.pa_pages_resize(tables, ld, i32([30, 0]), refs, caches, 16)
    status(ws)
    ws = binding.pa_pages_resize(tables, ld, i32([64, 0]), refs, caches, 16)
    status(ws)
    assert p.resize([30, 0]) and p.resize([64, 0])
    p.equals(tables, ld, refs, caches)


def test_bad_rows_are_recorded_and_left():
    p = Pool(5, [30, 20, 16], 4, 40, 16)
    bad = binding.PA_ERR_DEVICE_BOUNDS
    for new, lens in (([30, -1, 16], None), ([30, 65, 16], None), ([30, 20, 16], [30, -2, 16]),
                      ([30, 20, 16], [30, 99, 16])):
        tables, ld, refs, caches = p.on_gpu()
        if lens:
            ld = i32(lens)
        before = ld.tolist()
        ws = binding.pa_pages_resize(tables, ld, i32(new), refs, caches, 16)
        status(ws, bad)
        assert ld.tolist() == before and refs.tolist() == p.refs and torch.equal(tables.cpu(), p.tables)
    # An id outside the pool in a partly filled block: that row is left, the others go on.
    tables, ld, refs, caches = p.on_gpu()
    tables[0, 1] = 40
    ws = binding.pa_pages_resize(tables, ld, i32([17, 0, 16]), refs, caches, 16)
    status(ws, bad)
    assert ld.tolist() == [30, 0, 16]
    # ... and among the blocks given back: counted nowhere.
    tables, ld, refs, caches = p.on_gpu()
    tables[1, 1] = -3
    ws = binding.pa_pages_resize(tables, ld, i32([30, 0, 16]), refs, caches, 16)
    status(ws, bad)
    want = list(p.refs)
    want[int(p.tables[1, 0])] -= 1
    assert refs.tolist() == want and ld.tolist() == [30, 0, 16]
    # A count that is 0 already stays 0.
    tables, ld, refs, caches = p.on_gpu()
    refs[int(p.tables[2, 0])] = 0
    ws = binding.pa_pages_resize(tables, ld, i32([30, 20, 0]), refs, caches, 16)
    status(ws, bad)
    assert int(refs.min()) == 0
    # Forks of parents that do not exist, or with a bad length, are empty rows.
    tables, ld, refs, caches = p.on_gpu()
    ld[1] = 1000
    out, lo = torch.full((4, 4), -5, dtype=torch.int32, device="cuda"), i32([9] * 4)
    ws = binding.pa_pages_fork(out, lo, tables, ld, i32([3, 1, -2, 0]), refs, caches, 16)
    status(ws, bad)
    assert lo.tolist() == [0, 0, 0, 30] and bool((out[:3] == -5).all())
    # Compaction: a table that holds a free block, or none of the pool's.
    for v in (1000, -1, None):
        tables, ld, refs, caches = p.on_gpu()
        if v is None:
            v = max(b for b in range(40) if p.refs[b] == 0 and b >= sum(x > 0 for x in p.refs))
        tables[2, 0] = v
        ws = binding.pa_pages_compact(tables, ld, refs, caches, 16)
        status(ws, bad)
        assert int(tables[2, 0]) == v


def test_many_caches_of_odd_page_sizes():
    """More caches than one launch takes; pages from 16 bytes to several copy steps."""
    r = random.Random(6)
    p = Pool(6, [50, 7, 33], 5, 30, 16, caches=[(r.choice([1, 2, 5, 300, 700]),) for _ in range(131)])
    tables, ld, refs, caches = p.on_gpu()
    out, lo = torch.zeros((4, 5), dtype=torch.int32, device="cuda"), i32([0] * 4)
    ws = binding.pa_pages_fork(out, lo, tables, ld, i32([0, 1, 2, 0]), refs, caches, 16)
    status(ws)
    want, wl = torch.zeros((4, 5), dtype=torch.int32), [0] * 4
    assert p.fork([0, 1, 2, 0], want, wl)
    p.equals(tables, ld, refs, caches)
    ws = binding.pa_pages_resize(tables, ld, i32([0, 7, 33]), refs, caches, 16)
    status(ws)
    assert p.resize([0, 7, 33])
    p.tables, p.lens = torch.cat([p.tables, want]), p.lens + wl
    tables, ld = torch.cat([tables, out]), torch.cat([ld, lo])
    ws = binding.pa_pages_compact(tables, ld, refs, caches, 16)
    status(ws)
    p.compact()
    p.equals(tables, ld, refs, caches)


def test_no_caches_no_rows_and_unaligned_counts():
    p = Pool(7, [30, 20], 4, 40, 16, caches=())
    tables, ld, refs, _ = p.on_gpu()
    wide = torch.zeros(41, dtype=torch.int32, device="cuda")
    wide[1:] = refs
    refs = wide[1:]  # 4 bytes past a 16-byte boundary
    status(binding.pa_pages_resize(tables, ld, i32([35, 3]), refs, [], 16))
    assert p.resize([35, 3])
    p.equals(tables, ld, refs, [])
    status(binding.pa_pages_compact(tables, ld, refs, [], 16))
    p.compact()
    p.equals(tables, ld, refs, [])
    empty = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    status(binding.pa_pages_fork(empty.clone(), i32([]), tables, ld, i32([]), refs, [], 16))
    status(binding.pa_pages_resize(empty, i32([]), i32([]), refs, [], 16))
    p.equals(tables, ld, refs, [])


def test_replays_from_a_cuda_graph():
    """A resize and its undoing, captured once: every replay gives the same pool."""
    p = Pool(8, [30, 100, 64, 5], 9, 60, 16, share=2)
    tables, ld, refs, caches = p.on_gpu()
    up, back = i32([47, 20, 65, 0]), i32([30, 20, 64, 0])
    ws = torch.empty(binding.pages_workspace_bytes(4, 9, 60), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty_like(ws)  # each captured call with a status of its own

    def call():
        binding.pa_pages_resize(tables, ld, up, refs, caches, 16, workspace=ws)
        binding.pa_pages_resize(tables, ld, back, refs, caches, 16, workspace=ws2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for v in (up.tolist(), back.tolist()):
        assert p.resize(v)
    p.equals(tables, ld, refs, caches)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        status(ws)
        status(ws2)
        for v in (up.tolist(), back.tolist()):
            assert p.resize(v)
        p.equals(tables, ld, refs, caches)


def test_refusals():
    p = Pool(9, [30, 20], 4, 40, 16)
    tables, ld, refs, caches = p.on_gpu()
    with pytest.raises(ValueError):
        binding.pa_pages_resize(tables, ld, i32([1]), refs, caches, 16)
    with pytest.raises(TypeError):
        binding.pa_pages_resize(tables, ld, torch.tensor([1, 2], device="cuda"), refs, caches, 16)
    with pytest.raises(ValueError):
        binding.pa_pages_resize(tables, ld, i32([1, 2]), refs, [c[:5] for c in caches], 16)
    with pytest.raises(ValueError):
        binding.pa_pages_resize(tables, ld, i32([1, 2]), refs, [c.cpu() for c in caches], 16)
    with pytest.raises(binding.PaError):  # pages that are no multiple of 16 bytes
        binding.pa_pages_resize(tables, ld, i32([1, 2]), refs, [caches[0][:, :24].contiguous()], 16)
    with pytest.raises(binding.PaError):  # the children's rows lie in the parents'
        binding.pa_pages_fork(tables, i32([0, 0]), tables, ld, i32([0, 1]), refs, caches, 16)
    with pytest.raises(binding.PaError):
        binding.pa_pages_compact(tables, ld, refs, caches, 16, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.PaError):
        binding.pa_pages_compact(tables, ld, refs, caches, 0)
    p.equals(tables, ld, refs, caches)


def test_new_lengths_that_are_the_lengths():
    """A resize to the lengths themselves (the same array) changes nothing."""
    p = Pool(10, [30, 20, 0, 64], 4, 40, 16)
    tables, ld, refs, caches = p.on_gpu()
    status(binding.pa_pages_resize(tables, ld, ld, refs, caches, 16))
    assert p.resize(list(p.lens))
    p.equals(tables, ld, refs, caches)
    with pytest.raises(binding.PaError):  # an array that is the lengths' but for the first
        both = i32([30, 20, 0, 64, 64])
        binding.pa_pages_resize(tables, both[:4], both[1:], refs, caches, 16)
    with pytest.raises(binding.PaError):  # parents in the array that takes the children's lengths
        out = torch.zeros((4, 4), dtype=torch.int32, device="cuda")
        par = i32([0, 1, 2, 3])
        binding.pa_pages_fork(out, par, tables, ld, par, refs, caches, 16)
    p.equals(tables, ld, refs, caches)


def test_an_unchanged_length_in_a_shared_block_gets_a_copy():
    """Rows that end in a partly filled block that others hold: a copy each, at the same length
    too; a row that ends on a block's edge, or holds its last block alone, is left as it is."""
    p = Pool(11, [24, 24, 32, 24, 7], 4, 30, 16)
    for s in (1, 3):  # rows 0, 1 and 3 hold the same two blocks
        for j in range(2):
            p.refs[int(p.tables[s, j])] -= 1
            p.tables[s, j] = p.tables[0, j]
            p.refs[int(p.tables[0, j])] += 1
    tables, ld, refs, caches = p.on_gpu()
    shared, before = int(p.tables[0, 1]), p.tables.clone()
    status(binding.pa_pages_resize(tables, ld, i32([24, 24, 32, 24, 7]), refs, caches, 16))
    assert p.resize([24, 24, 32, 24, 7])
    p.equals(tables, ld, refs, caches)
    last = [int(tables[s, 1]) for s in (0, 1, 3)]
    assert len({shared, *last}) == 4 and refs[shared] == 0 and all(refs[b] == 1 for b in last)
    assert all(torch.equal(c[shared], c[b]) for c in caches for b in last)
    assert torch.equal(tables[2].cpu(), before[2]) and torch.equal(tables[4].cpu(), before[4])
    # Now each holds its own: the same call again changes nothing.
    status(binding.pa_pages_resize(tables, ld, i32([24, 24, 32, 24, 7]), refs, caches, 16))
    p.equals(tables, ld, refs, caches)


def test_every_holder_cut_back_needs_a_block_of_its_own():
    """Two rows cut back into the block that they alone share: two copies, so a pool with one
    free block refuses both at once and takes them one after the other."""
    p = Pool(12, [32, 32], 3, 4, 16, share=2)
    assert sum(x == 0 for x in p.refs) == 2
    p.refs[[b for b in range(4) if p.refs[b] == 0][0]] = 1  # (someone else's)
    tables, ld, refs, caches = p.on_gpu()
    status(binding.pa_pages_resize(tables, ld, i32([20, 20]), refs, caches, 16), binding.PA_ERR_NO_BLOCKS)
    p.equals(tables, ld, refs, caches)
    for new in ([20, 32], [20, 20]):
        status(binding.pa_pages_resize(tables, ld, i32(new), refs, caches, 16))
        assert p.resize(new)
        p.equals(tables, ld, refs, caches)
