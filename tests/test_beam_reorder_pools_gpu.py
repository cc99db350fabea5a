"""Reordering where a pool is too small: rows that get no room keep their tokens, whatever the others go on to store."""

import pytest
import torch

import bit_matmul_amd as bm
from tests.test_beam_reorder_gpu import layers_of

pytestmark = pytest.mark.gpu
PAGE, D = 16, 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bm.lib()
    yield
    torch.cuda.synchronize()


class Rows:
    """The rows of groups of beams, and the tokens (whole numbers below 128) that each should hold."""

    def __init__(self, table, histories, groups, num_pages, first, each):
        self.layers = layers_of(2, num_pages, PAGE, 1, D, 32, seed=num_pages)
        self.table, self.histories, self.groups, self.pool = table.cuda(), histories, groups, dict(first_page=first, pages_per_group=each)
        self.lens = torch.tensor([len(h) for h in histories], dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tokens = [t for h in histories for t in h]
        self.store(tokens, self.places())

    def places(self):
        return torch.cat([self.table[r, j // PAGE].long() * PAGE + j % PAGE for r, h in enumerate(self.histories)
                          for j in [torch.arange(len(h), device="cuda")]])

    def store(self, tokens, slots):
        x = torch.tensor(tokens, dtype=torch.bfloat16, device="cuda").view(-1, 1, 1).expand(-1, 1, D).contiguous()
        for i, c in enumerate(self.layers.caches):
            bm.bitmm_kv_append(x + i, x - i, slots, c)

    def step(self, parents, tokens):
        """One reorder and append, and a look at all that the rows then hold. Returns their slots."""
        p = torch.tensor(parents, dtype=torch.int32, device="cuda").view(self.groups, -1)
        self.table, self.lens, slots = bm.kv_beam_reorder(self.layers, self.table, self.lens, p, status=self.status, **self.pool)
        beams, at = p.shape[1], slots.tolist()
        self.histories = [(self.histories[r // beams * beams + q] if q >= 0 else []) + ([t] if at[r] >= 0 else [])
                          for r, (q, t) in enumerate(zip(parents, tokens))]
        self.store(tokens, slots)
        assert self.lens.tolist() == [len(h) for h in self.histories]
        want = torch.tensor([t for h in self.histories for t in h], device="cuda").view(-1, 1, 1).expand(-1, 1, D)
        for i, c in enumerate(self.layers.caches):
            k, v = bm.kv_read(c, self.places(), dtype=torch.float16)
            assert torch.equal(k.long(), want + i) and torch.equal(v.long(), want - i)
        return at


def test_a_page_that_a_longer_row_goes_on():
    """Two rows of one partly filled page, with no page for the second: later the longer one has it, wherever it stands."""
    for swaps in ([[1, 0]], [[0, 1], [1, 0], [1, 0]], [[1, 0], [0, 1], [0, 1]]):
        shared = [t % 100 for t in range(20)]
        rows = Rows(torch.tensor([[4, 7, 0]] * 2, dtype=torch.int32), [shared, shared], 1, 12, 7, 1)
        assert rows.step([0, 1], [101, 102]) == [7 * PAGE + 4, -1]
        for i, parents in enumerate(swaps):
            lens = rows.lens.tolist()
            longer = max(range(2), key=lambda r: lens[parents[r]])
            slots = rows.step(parents, [103 + 2 * i, 104 + 2 * i])
            assert slots[longer] >= 0 and slots[1 - longer] == -1
    assert rows.status.item() == 1


def test_equal_rows_and_more_than_two():
    """Of rows with as many tokens the first keeps the page; shorter ones before them do not."""
    shared = [t % 100 for t in range(20)]
    histories = [shared[:18], shared, shared[:19], shared]
    rows = Rows(torch.tensor([[4, 7, 0]] * 4, dtype=torch.int32), histories, 1, 12, 7, 3)
    assert rows.step([0, 1, 2, 3], [101, 102, 103, 104]) == [8 * PAGE + 2, 7 * PAGE + 4, 9 * PAGE + 3, -1]


@pytest.mark.parametrize("each", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("beams", [2, 3, 8])
def test_searches_on_small_pools(beams, each):
    """Many steps of random parents over pools that end, after prompts whose last page is not full. Every row's tokens
    are its history after each."""
    groups, width, first = 2, 5, 4
    g = torch.Generator().manual_seed(10 * beams + each)
    prompt = [torch.randint(0, 100, (n,), generator=g).tolist() for n in (21, 9)]
    table = torch.zeros(groups * beams, width, dtype=torch.int32)
    for r in range(groups * beams):
        table[r, :2] = torch.tensor([[0, 1], [2, 3]][r // beams])
    rows = Rows(table, [list(prompt[r // beams]) for r in range(groups * beams)], groups, first + groups * each + 3, first, each)
    for i in range(60):
        parents = torch.randint(-1 if i % 20 == 19 else 0, beams, (groups * beams,), generator=g)
        if i % 3 == 0:
            parents = torch.cat([torch.randperm(beams, generator=g) for _ in range(groups)])
        rows.step(parents.tolist(), torch.randint(0, 100, (groups * beams,), generator=g).tolist())
