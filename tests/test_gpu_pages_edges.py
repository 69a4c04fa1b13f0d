"""The pages of the cache where a batch has gaps or no rows, and where a page is as
large as it can be: against the rules of the book-keeping."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


def pool(rows, cols, pages):
    return (torch.full((rows, cols), -1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda"),
            torch.zeros(pages, dtype=torch.int32, device="cuda"))


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("ends,total", [((3, 13, 13, 20), 32), ((0, 10, 10, 17), 17), ((0, 0, 0, 0), 9), ((5, 5, 25, 30), 31)])
@pytest.mark.parametrize("on_side", [False, True])
def test_entries_of_no_row_store_nothing(ends, total, on_side):
    # a padded batch of prompts: what the allocator hands out again is full of slots of earlier calls
    page, pages, hkv, d = 16, 12, 2, 64
    table, lens, refs = pool(3, 4, pages)
    caches = [torch.full((pages * page, hkv * d), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream() if on_side else None
    for _ in range(4):
        old = [torch.full((total,), pages * page - 1, dtype=torch.int32, device="cuda") for _ in range(8)]
        del old
        table.fill_(-1), lens.zero_(), refs.zero_()
        torch.cuda.synchronize()
        slots, info = fp8rl.kv_reserve(table, lens, refs, page, caches, cu_seqlens=ints(*ends), total_tokens=total, stream=side)
        torch.cuda.synchronize()
        want, at = [-1] * total, 0
        for r in range(3):
            for i in range(ends[r + 1] - ends[r]):
                want[ends[r] + i] = (at + i // page) * page + i % page
            at += -(-(ends[r + 1] - ends[r]) // page)
        assert slots.tolist() == want and info.tolist() == [pages - at, 0]
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(total, h, d, generator=g, device="cuda").bfloat16() for h in (4, hkv, hkv))
    fp8rl.rotary_kv_append(q, k, v, torch.zeros(total, dtype=torch.int32, device="cuda"), fp8rl.rotary_freqs(d), slots, *caches,
                           torch.full((2,), 0.01, device="cuda"))
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots[slots >= 0].long()] = False
    assert all((c[rest] == 0x55).all() for c in caches)


@pytest.mark.parametrize("pages,free", [(5, 5), (0, 0), (70001, 69997)])
def test_an_empty_batch_reports_the_free_pages(pages, free):
    table, lens, refs = pool(0, 4, pages)
    refs[:pages - free] = 2
    for more in ({}, {"cu_seqlens": ints(0), "total_tokens": 3}, {"out": (torch.empty(0, dtype=torch.int32, device="cuda"), ints(7, 7))},
                 {"stream": torch.cuda.Stream()}, {"workspace": torch.empty(4096, dtype=torch.uint8, device="cuda")}):
        old = [torch.full((2,), -9, dtype=torch.int32, device="cuda") for _ in range(8)]
        del old
        torch.cuda.synchronize()
        slots, info = fp8rl.kv_reserve(table, lens, refs, 16, **more)
        torch.cuda.synchronize()
        assert info.tolist() == [free, 0] and slots.tolist() == [-1] * more.get("total_tokens", 0)
    assert int(refs.sum()) == 2 * (pages - free)


def test_ranges_that_begin_ahead_of_the_entries():
    # clamped to the entries there are: the first of them is the row's first new token
    table, lens, refs = pool(2, 4, 10)
    lens[0] = 5
    table[0, 0], refs[0] = 0, 1
    slots, info = fp8rl.kv_reserve(table, lens, refs, 16, cu_seqlens=ints(-3, 4, 9), total_tokens=7)
    assert slots.tolist() == [5, 6, 7, 8, 16, 17, 18] and info.tolist() == [8, 0] and lens.tolist() == [9, 3]
    slots, _ = fp8rl.kv_reserve(table, lens, refs, 16, count=ints(2, 1), cu_seqlens=ints(-2 ** 31, 3, 2 ** 31 - 1), total_tokens=5)
    assert slots.tolist() == [9, 10, -1, 19, -1] and lens.tolist() == [11, 4]


@pytest.mark.parametrize("width", [2 ** 31 - 1, 2 ** 31 - 1024])
def test_a_page_as_large_as_it_can_be(width):
    # byte numbers within a page end at 2^31: odd widths go byte by byte, others by 16-byte pieces
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    cache = torch.zeros(3, width, dtype=torch.uint8, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    cache[2, :4096] = torch.randint(1, 255, (4096,), generator=g, device="cuda", dtype=torch.int64).to(torch.uint8)
    cache[2, -4096:] = torch.randint(1, 255, (4096,), generator=g, device="cuda", dtype=torch.int64).to(torch.uint8)
    cache[2, width // 2] = 7
    cache[1] = 9
    table, lens, refs = ints(2, -1, 1, -1).view(2, 2), ints(1, 1), ints(0, 1, 1)
    assert int(fp8rl.kv_compact(table, lens, refs, 1, [cache])) == 2
    assert table[:, 0].tolist() == [0, 1] and refs.tolist() == [1, 1, 0]
    assert torch.equal(cache[0], cache[2]) and bool((cache[1] == 9).all())
    del cache
    torch.cuda.empty_cache()
