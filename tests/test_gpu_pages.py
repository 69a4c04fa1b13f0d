"""The pages of the cache: reserve, fork and compact against a plain model of the
book-keeping on the host, and the contents they move byte for byte."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


def blocks(n, page):
    return -(-n // page)


class Model:
    """The book-keeping and the contents on the host."""

    def __init__(self, rows, cols, page, pages, width, n_caches, seed=0, ld=None, skip=0):
        self.page, self.cols = page, cols
        g = torch.Generator().manual_seed(seed)
        self.table = torch.full((rows, cols), -1, dtype=torch.int32)
        self.lens = torch.zeros(rows, dtype=torch.int32)
        self.refs = torch.zeros(pages, dtype=torch.int32)
        self.caches = [torch.randint(0, 256, (pages * page + skip, width), generator=g).to(torch.uint8) for _ in range(n_caches)]
        self.pages = pages
        self.dev = [t.cuda() for t in (self.table, self.lens, self.refs)]
        ld = ld or width
        self.dev_caches = []
        for c in self.caches:
            wide = torch.zeros(c.shape[0], ld, dtype=torch.uint8, device="cuda")
            wide[:, :width] = c.cuda()
            self.dev_caches.append(wide[:, :width])
        self.handle = fp8rl.KvCaches(self.dev_caches)

    def reserve(self, counts, ranges=None, total=None, on_device=True):
        """counts per row; ranges: (begin, end) per row of the slots, else one after the other, even."""
        rows = len(counts)
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        refs0 = self.refs.clone()
        slots, at, refused = {}, 0, 0
        for r, k in enumerate(counts):
            n = int(self.lens[r])
            held, after = blocks(n, self.page), blocks(n + k, self.page)
            if after > self.cols:
                refused += 1
                continue
            last = int(self.table[r, held - 1]) if k > 0 and n % self.page else -1
            shared = 0 <= last < self.pages and int(refs0[last]) > 1
            need = after - held + shared if k > 0 else 0
            at += need
            if need and at > len(free):
                refused += 1
                continue
            give = free[at - need:at]
            if shared:
                new = give.pop(0)
                self.refs[last] -= 1
                self.refs[new] += 1
                self.table[r, held - 1] = new
                for c in self.caches:
                    c[new * self.page:new * self.page + n % self.page] = c[last * self.page:last * self.page + n % self.page]
            for j, p in enumerate(give):
                self.table[r, held + j] = p
                self.refs[p] += 1
            for i in range(k):
                pos = n + i
                slots[r, i] = int(self.table[r, pos // self.page]) * self.page + pos % self.page
            self.lens[r] = n + k
        return slots, [int((self.refs == 0).sum()), refused]

    def same(self):
        for name, want, got in zip(("table", "lens", "refs"), (self.table, self.lens, self.refs), self.dev):
            assert torch.equal(got.cpu(), want), (name, (got.cpu() != want).nonzero()[:5])
        for i, (want, got) in enumerate(zip(self.caches, self.dev_caches)):
            assert torch.equal(got.cpu(), want), i

    def step(self, counts, width=1):
        """A call with counts (at most `width` entries a row)."""
        rows = len(counts)
        want, info = self.reserve(counts)
        slots, got = fp8rl.kv_reserve(*self.dev, self.page, self.handle, count=torch.tensor(counts, dtype=torch.int32, device="cuda"),
                                      total_tokens=rows * width)
        full = torch.full((rows, width), -1, dtype=torch.int32)
        for (r, i), s in want.items():
            full[r, i] = s
        assert got.tolist() == info
        assert torch.equal(slots.cpu().view(rows, width), full)
        self.same()

    def prompts(self, counts, gap=0):
        ends = [gap]
        for k in counts:
            ends.append(ends[-1] + k)
        want, info = self.reserve(counts)
        total = ends[-1] + gap
        out = (torch.full((total,), -9, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"))
        slots, got = fp8rl.kv_reserve(*self.dev, self.page, self.handle, cu_seqlens=torch.tensor(ends, dtype=torch.int32, device="cuda"),
                                      total_tokens=total, out=out)
        full = torch.full((total,), -9, dtype=torch.int32)
        full[gap:ends[-1]] = -1
        for (r, i), s in want.items():
            full[ends[r] + i] = s
        assert got.tolist() == info
        assert torch.equal(slots.cpu(), full)
        self.same()

    def fork(self, parent, in_place=False):
        def holds(t, n):
            return [int(p) for p in t[:blocks(int(n), self.page)] if 0 <= int(p) < self.pages]

        old_t, old_l = self.table, self.lens
        new_t = torch.full((len(parent), self.cols), -1, dtype=torch.int32)
        new_l = torch.zeros(len(parent), dtype=torch.int32)
        for t, n in zip(old_t, old_l):
            for p in holds(t, n):
                self.refs[p] -= 1
        for i, p in enumerate(parent):
            if not 0 <= p < len(old_l) or (in_place and p != i and parent[p] != p):
                continue
            n = blocks(int(old_l[p]), self.page)
            new_t[i, :n] = old_t[p, :n]
            if in_place and p == i:
                new_t[i] = old_t[i]
            new_l[i] = old_l[p]
            for q in holds(old_t[p], old_l[p]):
                self.refs[q] += 1
        self.table, self.lens = new_t, new_l
        dev_parent = torch.tensor(parent, dtype=torch.int32, device="cuda")
        out = tuple(self.dev[:2]) if in_place else None
        t, l = fp8rl.kv_fork(*self.dev, dev_parent, self.page, out=out)
        self.dev = [t, l, self.dev[2]]
        self.same()

    def compact(self):
        used = [p for p in range(self.pages) if self.refs[p] > 0]
        n = len(used)
        src = [p for p in used if p >= n]
        dst = [p for p in range(n) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for c in self.caches:
            c0 = c.clone()
            for s, d in to.items():
                c[d * self.page:(d + 1) * self.page] = c0[s * self.page:(s + 1) * self.page]
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s].clone(), 0
        for r in range(len(self.lens)):
            for j in range(blocks(int(self.lens[r]), self.page)):
                self.table[r, j] = to.get(int(self.table[r, j]), int(self.table[r, j]))
        assert fp8rl.kv_compact(*self.dev, self.page, self.handle).tolist() == [n]
        self.same()


@pytest.mark.parametrize("page,width,n_caches,ld", [(16, 1024, 2, None), (1, 64, 1, None), (48, 80, 3, 96), (16, 70, 2, 75), (64, 256, 5, 512), (3, 16, 2, None)])
def test_a_rollout_of_random_steps(page, width, n_caches, ld):
    import random
    rng = random.Random(page)
    rows, cols, pages = 24, 9, 90
    m = Model(rows, cols, page, pages, width, n_caches, ld=ld)
    m.prompts([rng.randint(0, 4 * page) if r < 6 else 0 for r in range(rows)])
    m.fork([r % 6 if rng.random() < 0.8 else -1 for r in range(rows)])
    for _ in range(6):
        m.step([rng.randint(0, 1) for _ in range(rows)])
        m.step([rng.randint(0, page) for _ in range(rows)], width=page)
        m.fork([r if rng.random() < 0.7 else rng.randint(-2, rows) for r in range(rows)])
        m.compact()
        m.fork([r if rng.random() < 0.7 else -1 for r in range(rows)], in_place=True)
        m.prompts([rng.randint(0, 2 * page) if int(n) == 0 else 0 for n in m.lens], gap=2)
    m.fork([-1] * rows)
    assert not m.refs.any() and not m.lens.any()
    m.compact()


def test_all_who_share_a_page_write():
    m = Model(8, 4, 16, 40, 128, 2)
    m.prompts([21] + [0] * 7)
    m.fork([0] * 8)
    assert m.refs.max() == 8
    m.step([1] * 8)
    assert m.refs[m.table[:, 1].long()].max() == 1 and (m.refs == 0).sum() == 40 - 1 - 8
    m.step([1] * 8)


def test_a_full_last_page_is_not_copied():
    m = Model(4, 4, 16, 20, 64, 1)
    m.prompts([32, 0, 0, 0])
    m.fork([0, 0, 0, -1])
    m.step([1, 0, 1, 1])
    assert int(m.refs[m.table[0, 1].long()]) == 3


def test_refusals_leave_rows_alone():
    m = Model(6, 3, 16, 7, 64, 1)
    m.prompts([16, 16, 16, 0, 0, 0])
    m.step([1, 40, 1, 1, 33, 0], width=40)   # row 1 passes the table's end, row 4 the pages
    m.step([0, 0, 0, 30, 0, 0], width=48)
    m.step([1, 1, 1, 1, 1, 1])
    m.step([0] * 6)
    m.prompts([0, 0, 0, 0, 5, 60])


def test_no_pages_no_tokens_no_rows():
    m = Model(3, 2, 16, 0, 64, 1)
    m.step([1, 0, 1])
    m.fork([2, 1, 0])
    m.compact()
    m = Model(3, 0, 16, 5, 64, 1)
    m.step([1, 0, 1])
    m.fork([2, 1, 0])
    m.fork([-1, 1, 0], in_place=True)
    m.compact()
    m = Model(3, 2, 16, 5, 64, 0)
    m.step([1, 0, 1])
    m.prompts([0, 0, 0])
    m.compact()
    e = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    refs = torch.zeros(5, dtype=torch.int32, device="cuda")
    t, n = fp8rl.kv_fork(e, z, refs, torch.tensor([0, -1], dtype=torch.int32, device="cuda"), 16)
    assert t.tolist() == [[-1] * 4] * 2 and n.tolist() == [0, 0]
    assert fp8rl.kv_reserve(e, z, refs, 16)[0].shape == (0,)


@pytest.mark.parametrize("pages", [40000, 300001])
def test_many_pages_and_rows(pages):
    # a cluster plans; without contents on the host model's side but small ones
    rows, cols, page = 3000, 40, 4
    g = torch.Generator().manual_seed(pages)
    m = Model(rows, cols, page, pages, 16, 1)
    m.prompts([int(v) for v in torch.randint(0, 12, (rows,), generator=g)])
    # spread the used pages: free two rows in three, take more, free again
    m.fork([r if r % 3 == 0 else -1 for r in range(rows)])
    m.step([int(v) for v in torch.randint(0, 2, (rows,), generator=g)])
    m.fork([int(v) for v in torch.randint(-1, rows, (rows,), generator=g)])
    m.step([int(v) for v in torch.randint(0, 9, (rows,), generator=g)], width=8)
    m.compact()


def test_one_long_prompt():
    m = Model(2, 9000, 16, 9000, 16, 1)
    m.prompts([100003, 17])
    m.step([1, 1])


def test_counts_past_their_entries_and_odd_arguments():
    # counts are clamped to the entries, lengths to the table, entries outside the pages stand for none
    m = Model(3, 3, 8, 9, 32, 1)
    table, lens, refs = m.dev
    slots, info = fp8rl.kv_reserve(table, lens, refs, 8, m.handle, count=torch.tensor([5, -3, 2], dtype=torch.int32, device="cuda"), total_tokens=6)
    assert slots.view(3, 2).tolist() == [[0, 1], [-1, -1], [8, 9]] and info.tolist() == [7, 0]
    table[0, 0] = 1000
    lens[1] = 1000
    lens[2] = -5
    slots, info = fp8rl.kv_reserve(table, lens, refs, 8, m.handle)
    assert slots.tolist()[1:] == [-1, 16] and info.tolist() == [6, 1]
    assert int(lens[1]) == 1000


def test_attention_over_forked_and_compacted_pages_is_unchanged():
    hq, hkv, d, page, rows, cols, pages = 8, 2, 128, 16, 6, 8, 64
    g = torch.Generator("cuda").manual_seed(3)
    caches = [torch.randint(0, 120, (pages * page, hkv * d), generator=g, device="cuda", dtype=torch.int64).to(torch.uint8) for _ in range(2)]
    table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 50, 63, 63, 160, 161, 200], dtype=torch.int32, device="cuda")
    fp8rl.kv_reserve(table, lens, refs, page, caches, cu_seqlens=cu, total_tokens=200)
    q = torch.randn(rows, hq, d, generator=g, device="cuda").bfloat16()
    scales = torch.full((2,), 0.01, device="cuda")
    want = fp8rl.attn_decode(q, *caches, table, lens, scales, page)
    parent = torch.tensor([3, 0, 1, 3, 5, 3], dtype=torch.int32, device="cuda")
    table, lens = fp8rl.kv_fork(table, lens, refs, parent, page)
    p = parent.long()
    got = fp8rl.attn_decode(q[p].contiguous(), *caches, table, lens, scales, page)
    assert torch.equal(got[0], want[0][p])
    used = int(fp8rl.kv_compact(table, lens, refs, page, caches))
    assert used == int((refs > 0).sum()) and int(table.max()) < used
    assert not refs[used:].any()
    got = fp8rl.attn_decode(q[p].contiguous(), *caches, table, lens, scales, page)
    assert torch.equal(got[0], want[0][p])
    # a row that grows gets the shared page's contents; the others keep theirs
    slots, _ = fp8rl.kv_reserve(table, lens, refs, page, caches, count=torch.tensor([1, 0, 0, 0, 0, 0], dtype=torch.int32, device="cuda"))
    after = lens.clone()
    after[0] -= 1
    got = fp8rl.attn_decode(q[p].contiguous(), *caches, table, after, scales, page)
    assert torch.equal(got[0], want[0][p]) and slots.tolist()[1:] == [-1] * 5


def test_captured_steps_on_another_stream():
    m, n = (Model(5, 6, 16, 30, 256, 2) for _ in range(2))
    for x in (m, n):
        x.prompts([30, 20, 0, 0, 0])
        x.fork([0, 1, 0, 1, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, info = fp8rl.kv_reserve(*n.dev, n.page, n.handle)
    for _ in range(20):
        graph.replay()
        m.step([1] * 5)
        assert all(torch.equal(a, b) for a, b in zip(m.dev, n.dev))
        assert all(torch.equal(a, b) for a, b in zip(m.dev_caches, n.dev_caches))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want, want_info = m.reserve([1] * 5)
    slots, info = fp8rl.kv_reserve(*m.dev, m.page, m.handle, stream=side)
    side.synchronize()
    assert slots.tolist() == [want[r, 0] for r in range(5)] and info.tolist() == want_info
    m.same()


def test_pages_past_2_31_bytes():
    # slots stay 32-bit numbers, byte offsets do not
    page, width, pages = 16, 4096, 60000  # 3.9 GB
    cache = torch.empty(pages * page, width, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, -1], [pages - 2, -1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 16], dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[-2:] = 1
    refs[-1] = 2
    content = torch.randint(0, 255, (2 * page, width), device="cuda", dtype=torch.int64).to(torch.uint8)
    cache[-2 * page:] = content
    slots, info = fp8rl.kv_reserve(table, lens, refs, page, [cache])
    assert slots.tolist() == [5, page] and info.tolist() == [pages - 4, 0]
    assert torch.equal(cache[:5], content[page:page + 5])
    lens2 = torch.tensor([5, 16], dtype=torch.int32, device="cuda")
    table2 = torch.tensor([[pages - 1, -1], [pages - 2, -1]], dtype=torch.int32, device="cuda")
    refs.zero_()
    refs[-2:] = 1
    assert int(fp8rl.kv_compact(table2, lens2, refs, page, [cache])) == 2
    assert table2[:, 0].tolist() == [1, 0]
    assert torch.equal(cache[:2 * page], content)


def test_odd_places_and_strides():
    # arrays that start anywhere and a table that is a part of a wider one
    page, pages, rows, cols = 16, 70, 5, 6
    base = torch.zeros(pages + 3, dtype=torch.int32, device="cuda")
    wide = torch.full((rows, cols + 3), -7, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")[1:]
    table, refs = wide[:, 1:cols + 1], base[1:pages + 1]
    table.fill_(-1)
    pool = torch.randint(0, 255, (pages * page + 1, 96), device="cuda", dtype=torch.int64).to(torch.uint8)
    cache = pool[:, 1:65]  # no 16-byte pieces
    before = pool.clone()
    cu = torch.tensor([0, 20, 20, 20, 20, 20], dtype=torch.int32, device="cuda")
    slots, info = fp8rl.kv_reserve(table, lens, refs, page, [cache], cu_seqlens=cu, total_tokens=20)
    assert slots.tolist() == list(range(20)) and info.tolist() == [pages - 2, 0]
    fp8rl.kv_fork(table, lens, refs, torch.tensor([0, 0, -1, 0, -1], dtype=torch.int32, device="cuda"), page, out=(table, lens))
    slots, info = fp8rl.kv_reserve(table, lens, refs, page, [cache], count=torch.tensor([0, 1, 1, 1, 0], dtype=torch.int32, device="cuda"))
    assert slots.tolist() == [-1, 2 * page + 4, 3 * page, 4 * page + 4, -1] and info.tolist() == [pages - 5, 0]
    assert torch.equal(cache[2 * page:2 * page + 4], before[page:page + 4, 1:65])
    fp8rl.kv_fork(table, lens, refs, torch.tensor([-1, 1, -1, -1, -1], dtype=torch.int32, device="cuda"), page, out=(table, lens))
    used = fp8rl.kv_compact(table, lens, refs, page, [cache])
    assert int(used) == 2 and table[1].tolist()[:2] == [0, 1] and refs.tolist() == [1, 1] + [0] * (pages - 2)
    assert torch.equal(cache[page:page + 4], before[page:page + 4, 1:65])
    assert base[0] == 0 and not base[pages + 1:].any() and (wide[:, 0] == -7).all() and (wide[:, cols + 1:] == -7).all()
    assert torch.equal(pool[:, 0], before[:, 0]) and torch.equal(pool[:, 65:], before[:, 65:])


def test_two_streams_at_once():
    models = [Model(40, 12, 16, 400, 256, 4, seed=i) for i in range(2)]
    for m in models:
        m.prompts([21] + [0] * 39)
        m.fork([0] * 40)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(30):
        for m, s in zip(models, streams):
            with torch.cuda.stream(s):
                fp8rl.kv_reserve(*m.dev, m.page, m.handle)
    torch.cuda.synchronize()
    for m in models:
        for _ in range(30):
            m.reserve([1] * 40)
        m.same()


@pytest.mark.parametrize("entry", [-1, -7, 9, 2 ** 31 - 1, -2 ** 31, 2 ** 28])
def test_a_table_entry_that_is_no_page_has_no_slots(entry):
    # the tokens behind it on the same page have none either; those on the next page do
    m = Model(2, 3, 16, 9, 32, 1)
    m.prompts([13, 5])
    table, lens, refs = m.dev
    table[0, 0] = entry
    slots, info = fp8rl.kv_reserve(table, lens, refs, 16, m.handle, total_tokens=8)
    assert slots.tolist() == [-1, -1, -1, 32, 21, 22, 23, 24] and info.tolist() == [6, 0]
    table[0, 1] = entry
    cu = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    slots, info = fp8rl.kv_reserve(table, lens, refs, 16, m.handle, cu_seqlens=cu, total_tokens=3)
    assert slots.tolist() == [-1, -1, 25] and info.tolist() == [6, 0]


@pytest.mark.parametrize("width,ld", [(32, 32), (33, 40)])
def test_many_copies_at_once(width, ld):
    # several copies a CTA: runs of one page that begin and end anywhere, then moves of pages that differ
    m = Model(140, 4, 8, 700, width, 64, ld=ld)
    m.prompts([3 + 5 * (r % 5) for r in range(24)] + [0] * 116)
    parent, r = [], 0
    while len(parent) < 140:
        parent += [r % 24] * (1 + r % 9)
        r += 1
    m.fork(parent[:140])
    m.step([1] * 140)
    m.step([7] * 140, width=7)
    m.fork([r if r % 3 else -1 for r in range(140)])
    m.step([r % 4 for r in range(140)], width=3)
    m.compact()
