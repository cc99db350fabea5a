"""Reordering of the cached states on the GPU: tables, lengths, slots and every word of every page against a plain
form of the same rules, and whole searches whose every row's history is known."""

import pytest
import torch

import bit_matmul_amd as bm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


def layers_of(n, pages, page, heads, D, group, seed=0):
    """Caches whose every word is of its own."""
    g = torch.Generator().manual_seed(seed)
    caches = []
    for _ in range(n):
        sides = []
        for _ in range(2):
            sides += [torch.randint(-2 ** 31, 2 ** 31, (pages, heads, page, D // 8), generator=g).to(torch.int32).cuda(),
                      torch.randn(pages, heads, page, D // group, 2, generator=g).bfloat16().cuda()]
        caches.append(bm.KVCache(*sides))
    return bm.KVLayers(caches)


def tensors(layers):
    return [t for c in layers.caches for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]


def plain(table, lens, parents, page, num_pages, first, each):
    """(table, lens, slots, copies [(src, dst, tokens)], whether something was out of range) of lists."""
    groups, beams = len(parents), len(parents[0])
    width = len(table[0])
    new, new_lens, slots, copies, wrong = [list(r) for r in table], [], [], [], False
    for g in range(groups):
        rows = range(g * beams, (g + 1) * beams)
        base, held = first + g * each, set()
        n = {}
        for j, r in enumerate(rows):
            p = parents[g][j]
            if not -1 <= p < beams:
                wrong, p = True, -1
            n[r] = -1
            if p >= 0:
                length = lens[g * beams + p]
                n[r] = min(max(length, 0), width * page)
                wrong = wrong or n[r] != length
                for c in range(-(-n[r] // page)):
                    new[r][c] = table[g * beams + p][c]
                    held.add(new[r][c])
        free = [x for x in range(base, base + each) if x not in held]
        seen, table_at = set(), [list(r) for r in new]
        for r in rows:
            if n[r] < 0:
                new_lens.append(0)
                slots.append(-1)
                continue
            column, part = divmod(n[r], page)
            at = -1
            mine = base <= new[r][column] < base + each or not 0 <= new[r][column] < num_pages if part else False
            full = part and any(n[o] // page > column and table_at[o][column] == new[r][column] for o in rows)
            if full and 0 <= new[r][column] < num_pages:
                mine = False
            if part and mine and new[r][column] not in seen:
                seen.add(new[r][column])
                at = new[r][column] if 0 <= new[r][column] < num_pages else -1
            elif column < width and free:
                at = free.pop(0)
                if part and 0 <= new[r][column] < num_pages:
                    copies.append((new[r][column], at, part))
                elif part:
                    wrong = True
                new[r][column] = at
            wrong = wrong or at < 0
            new_lens.append(n[r] + (at >= 0))
            slots.append(at * page + part if at >= 0 else -1)
    return new, new_lens, slots, copies, wrong


def check(layers, table, lens, parents, first, each, in_place=False):
    page, num_pages = layers.page_size, layers.caches[0].num_pages
    want = plain(table.tolist(), lens.tolist(), parents.tolist(), page, num_pages, first, each)
    before = [t.clone() for t in tensors(layers)]
    for src, dst, tokens in want[3]:
        for t in before:
            t[dst, :, :tokens] = t[src, :, :tokens]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, n, p = table.cuda(), lens.cuda(), parents.cuda()
    if in_place:
        slots = torch.empty(lens.shape, dtype=torch.int64, device="cuda")
        ws = torch.empty(bm.bitmm_kv_beam_reorder_workspace_bytes(*parents.shape), dtype=torch.uint8, device="cuda")
        bm.bitmm_kv_beam_reorder(layers, t, n, p, t, n, slots, ws, first_page=first, pages_per_group=each, status=status)
        got = t, n, slots
    else:
        got = bm.kv_beam_reorder(layers, t, n, p, first_page=first, pages_per_group=each, status=status)
        assert torch.equal(t.cpu(), table) and torch.equal(n.cpu(), lens)
    for a, b in zip(got, want):
        assert a.tolist() == b
    assert status.item() == int(want[4])
    assert all(torch.equal(a, b) for a, b in zip(tensors(layers), before))
    return got


CASES = [  # groups, beams, layers, page, heads, dims, group, longest
    (1, 1, 1, 16, 1, 64, 32, 40), (1, 4, 3, 16, 8, 128, 64, 100), (5, 3, 2, 32, 3, 256, 128, 200), (2, 64, 1, 64, 2, 64, 64, 300),
    (9, 8, 70, 16, 1, 64, 64, 50), (3, 5, 4, 256, 5, 128, 32, 700), (40, 4, 2, 128, 2, 256, 32, 400), (1, 33, 130, 16, 2, 64, 32, 70),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_against_plain(case, in_place):
    groups, beams, n, page, heads, D, group, longest = case
    g = torch.Generator().manual_seed(longest)
    width = -(-longest // page) + 1
    each, first = beams * width, 2
    layers = layers_of(n, first + groups * each, page, heads, D, group, seed=longest)
    order = torch.stack([torch.randperm(each, generator=g) for _ in range(groups)]) + first + each * torch.arange(groups)[:, None]
    table = order.view(groups, beams, width)
    table = table.clone()
    table[:, :, :width // 2] = table[:, :1, :width // 2]   # early pages are everybody's
    table = table.view(groups * beams, width).to(torch.int32)
    for trial in range(4):
        one = torch.randint(width // 2 * page, longest + 1, (groups, 1), generator=g).expand(groups, beams)
        lens = one if trial % 2 == 0 else torch.randint(width // 2 * page, longest + 1, (groups, beams), generator=g)
        lens = lens.reshape(-1).to(torch.int32)
        parents = torch.randint(-1 if trial == 3 else 0, beams, (groups, beams), generator=g).to(torch.int32)
        check(layers, table, lens, parents, first, each, in_place)


def test_edges():
    """Empty rows, exactly filled pages, one token, rows that fill their table, everybody the same parent."""
    layers = layers_of(2, 40, 16, 2, 64, 32)
    table = torch.tensor([[1, 2, 3], [1, 5, 6], [1, 8, 9], [1, 11, 12]], dtype=torch.int32)
    same = torch.zeros(1, 4, dtype=torch.int32)
    own = torch.arange(4, dtype=torch.int32)[None]
    for lens in ([0, 0, 0, 0], [1, 1, 1, 1], [15, 15, 15, 15], [16, 16, 16, 16], [17, 32, 33, 47], [31, 0, 1, 16]):
        for parents in (same, own, own.flip(1), torch.tensor([[3, -1, 3, -1]], dtype=torch.int32), torch.full((1, 4), -1, dtype=torch.int32)):
            check(layers, table, torch.tensor(lens, dtype=torch.int32), parents, 1, 20)
    # 48 tokens fill the table: no place for another
    check(layers, table, torch.tensor([48, 48, 47, 48], dtype=torch.int32), own, 1, 20)


def test_beams_that_start_on_one_page():
    """After a prompt all rows are the same: the first keeps the partly filled page."""
    layers = layers_of(1, 40, 16, 2, 64, 32)
    table = torch.tensor([[4, 7, 0]] * 3, dtype=torch.int32)
    got = check(layers, table, torch.tensor([20, 20, 20], dtype=torch.int32), torch.arange(3, dtype=torch.int32)[None], 1, 30)
    assert got[0][:, 1].tolist() == [7, 1, 2]


def test_pages_of_a_prompt_are_not_written():
    """Rows whose partly filled page lies outside their pool all copy it."""
    layers = layers_of(2, 40, 16, 2, 64, 32)
    table = torch.tensor([[4, 7, 0]] * 3, dtype=torch.int32)
    got = check(layers, table, torch.tensor([20, 20, 20], dtype=torch.int32), torch.arange(3, dtype=torch.int32)[None], 10, 9)
    assert got[0][:, 1].tolist() == [10, 11, 12] and got[0][:, 0].tolist() == [4, 4, 4]


def test_a_pool_that_ends():
    layers = layers_of(1, 40, 16, 2, 64, 32)
    table = torch.tensor([[4, 7, 0]] * 4, dtype=torch.int32)
    lens = torch.tensor([20, 20, 20, 20], dtype=torch.int32)
    for each in (0, 1, 2, 3):
        for parents in (torch.arange(4, dtype=torch.int32)[None], torch.tensor([[-1, 2, 1, 0]], dtype=torch.int32)):
            check(layers, table, lens, parents, 10, each)
            check(layers, table, torch.tensor([16, 32, 16, 16], dtype=torch.int32), parents, 10, each)


def test_a_page_that_is_full_for_a_longer_row():
    """Where a pool ended, one row got no room and the other filled the page that both have: it is copied."""
    layers = layers_of(2, 40, 16, 2, 64, 32)
    table = torch.tensor([[4, 7, 0]] * 2, dtype=torch.int32)
    own = torch.tensor([[0, 1]], dtype=torch.int32)
    t, n, slots = check(layers, table, torch.tensor([31, 31], dtype=torch.int32), own, 7, 1)
    assert n.tolist() == [32, 31] and slots.tolist() == [7 * 16 + 15, -1]
    for order in (own, own.flip(1)):
        got = check(layers, t.cpu(), n.cpu(), order, 7, 9)
        at = order[0].tolist().index(1)
        assert got[0][at, 1].item() != 7 and got[0][1 - at, 1].item() == 7


def test_out_of_range():
    layers = layers_of(1, 40, 16, 2, 64, 32)
    table = torch.tensor([[4, 7, 0], [5, -1, 0], [6, 40, 1], [8, 2 ** 31 - 1, 1]], dtype=torch.int32)
    lens = torch.tensor([20, 20, 20, 18], dtype=torch.int32)
    own = torch.arange(4, dtype=torch.int32)[None]
    check(layers, table, lens, own, 10, 20)
    check(layers, table, lens, torch.tensor([[1, 1, 2, 2]], dtype=torch.int32), 10, 20)
    check(layers, table, lens, torch.tensor([[4, -2, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32), 10, 20)
    check(layers, table, torch.tensor([-1, 49, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32), own, 10, 20)


def test_large_pools_and_tables():
    """Pools of more than 64 words of bits, their first pages all held, and tables wider than a pass."""
    layers = layers_of(1, 9000, 16, 1, 64, 64)
    beams, width = 3, 1500
    table = torch.randperm(6000, generator=torch.Generator().manual_seed(1))[:beams * width].view(beams, width).to(torch.int32)
    table[0, :1400] = torch.arange(1400) + 5
    parents = torch.tensor([[2, 0, 0]], dtype=torch.int32)
    for lens in ([1400 * 16 - 3] * 3, [1499 * 16] * 3, [100, 23000, 5]):
        check(layers, table, torch.tensor(lens, dtype=torch.int32), parents, 5, 8990)


@pytest.mark.parametrize("beams, page, steps", [(4, 16, 60), (7, 32, 70), (1, 16, 40), (16, 16, 35)])
def test_searches(beams, page, steps):
    """Many steps in place, replayed from a graph: every row's tokens are its history, as they were appended."""
    groups, D = 3, 64
    width = -(-steps // page) + 1
    first, each = 4, beams * width
    layers = layers_of(2, first + groups * each, page, 1, D, 32, seed=beams)
    rows = groups * beams
    table = torch.zeros(rows, width, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    parents = torch.zeros(groups, beams, dtype=torch.int32, device="cuda")
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(bm.bitmm_kv_beam_reorder_workspace_bytes(groups, beams), dtype=torch.uint8, device="cuda")
    token = torch.zeros(rows, 1, D, dtype=torch.bfloat16, device="cuda")

    def step():
        bm.bitmm_kv_beam_reorder(layers, table, lens, parents, table, lens, slots, ws, first_page=first, pages_per_group=each, status=status)
        for i, c in enumerate(layers.caches):
            bm.bitmm_kv_append(token + i, token - i, slots, c, status=status)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    lens.zero_()
    g = torch.Generator().manual_seed(beams)
    histories = [[] for _ in range(rows)]
    for i in range(steps):
        p = torch.randint(0, beams, (groups, beams), generator=g)
        if i % 3 == 0:
            p = torch.arange(beams).expand(groups, beams)
        ids = torch.randint(0, 100, (rows,), generator=g)
        histories = [histories[r // beams * beams + p[r // beams, r % beams].item()] + [ids[r].item()] for r in range(rows)]
        parents.copy_(p)
        token.copy_(ids.view(-1, 1, 1).expand_as(token).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        if i % 7 == 0 or i == steps - 1:
            assert lens.tolist() == [len(h) for h in histories]
            n = i + 1
            j = torch.arange(n, device="cuda")
            at = table[:, j // page].long() * page + j % page
            assert at.shape == (rows, n)
            for l, c in enumerate(layers.caches):
                k, v = bm.kv_read(c, at.flatten().contiguous(), dtype=torch.float16)
                want = torch.tensor(histories, device="cuda").view(rows * n, 1, 1).expand(-1, 1, D)
                assert torch.equal(k.long(), want + l) and torch.equal(v.long(), want - l)
    assert status.item() == 0


def test_other_stream_and_launches():
    layers = layers_of(65, 40, 16, 2, 64, 32)
    table = torch.tensor([[4, 7, 0]] * 3, dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 20, 20], dtype=torch.int32, device="cuda")
    parents = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = bm.kv_beam_reorder(layers, table, lens, parents, first_page=10, pages_per_group=9, stream=stream)
    assert len(bm.bitmm_last_launches()) == 3   # the plan, and copies of up to 64 layers at a time
    torch.cuda.current_stream().wait_stream(stream)
    assert got[0].tolist() == [[4, 10, 0], [4, 11, 0], [4, 12, 0]] and got[2].tolist() == [164, 180, 196]
    c = layers.caches[64]
    assert torch.equal(c.k_codes[11, :, :4], c.k_codes[7, :, :4])
