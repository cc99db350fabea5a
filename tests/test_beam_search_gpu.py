"""examples/beam_search.py on the GPU: what its steps choose is what 64 bits choose from the same logits, the states that the
beams end with are their tokens', and captured steps are those run one by one."""

import importlib.util
import os

import pytest
import torch

import bit_matmul_amd as bm
from tests.test_beam_select_gpu import reference

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("beam_search", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def prompts(*lens, vocab=500):
    g = torch.Generator().manual_seed(sum(lens))
    return [torch.randint(0, vocab, (n,), generator=g).cuda() for n in lens]


def small(example, pages=120, page=16):
    return example.Model(500, 256, 2, 4, 1, 64, num_pages=pages, page_size=page)


def alone(example, model, prompt, tokens):
    """Sum of the log probabilities of tokens after a prompt, each predicted after all before it at once: the sequence
    through the layers as a prompt of its own."""
    whole = torch.cat([prompt, tokens[:-1]])
    other = example.Model(500, 256, 2, 4, 1, 64, num_pages=-(-len(whole) // 16), page_size=16)   # the same weights, an empty cache
    n = len(whole)
    at = torch.arange(n, device="cuda")
    table = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda")[None]
    cu, kv = torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    logits = other(whole, at.int(), at, lambda q, cache: bm.kv_attention(q, cache, table, kv, cu, max_q=n, max_kv=n),
                   last=slice(len(prompt) - 1, n))
    return torch.log_softmax(logits.double(), -1).gather(1, tokens[:, None].long()).sum().item()


@pytest.mark.parametrize("lens, beams, steps", [((40, 77), 4, 40), ((5,), 7, 33), ((130, 16, 1), 3, 20), ((700,), 16, 18)])
def test_scores_are_the_sequences(example, lens, beams, steps):
    """A beam's score against the same tokens as one sequence. Hidden states are bf16, rounded some ten times on the way, half a
    step of 2^-8 each: logits of a deviation of 2.5 are off by 2.5 sqrt(10) 2^-8 = 0.03 of one's deviation, and a key or value
    whose code falls on the other side for that adds less. A log probability is the difference of two such sums; 0.1 a step is
    three deviations for a single one, and a tenth of what one token's wrong states make: as much as the logits' own deviation."""
    model = small(example, pages=200)
    given = prompts(*lens)
    search = example.Search(model, given, beams, steps)
    tokens, scores = search.run(graph=False)
    assert model.status.item() == 0
    assert (scores[:, 1:] <= scores[:, :-1]).all() and scores.isfinite().all()
    for g, prompt in enumerate(given):
        assert len({tuple(t.tolist()) for t in tokens[g]}) == beams   # beams of one prompt are different sequences
        for b in range(beams):
            assert abs(alone(example, model, prompt, tokens[g, b]) - scores[g, b].item()) < 0.1 * steps


def test_each_choice(example):
    """The choices of every step, with an end that some beams reach, from the logits that they were made from."""
    model = small(example)
    search = example.Search(model, prompts(33, 60), 5, 25, end_token=7)
    seen, inner = [], model.__class__.__call__

    def spy(*a, **kw):
        logits = inner(model, *a, **kw)
        logits[:, 7] += 4   # a likely end
        seen.append((logits.clone(), search.scores.clone(), search.finished.clone()))
        return logits

    search.model = type("Spy", (), {"__call__": lambda self, *a, **kw: spy(*a, **kw), "caches": model.caches, "status": model.status})()
    for _ in range(24):
        search.step()
        logits, scores, finished = seen[-1]
        want = reference(logits, scores.view(-1), 5, 5, finished.view(-1), 7)
        assert torch.equal(search.parents.cpu().long(), want[1]) and torch.equal(search.tokens.cpu().long(), want[2])
        assert torch.equal(search.finished.cpu(), want[3])
    assert search.finished.any() and model.status.item() == 0


@pytest.mark.parametrize("lens, beams, steps", [((40, 77), 4, 40), ((300,), 2, 50)])
def test_captured_steps(example, lens, beams, steps):
    model, given = small(example), prompts(*lens)
    eager = example.Search(model, given, beams, steps).run(graph=False)
    for _ in range(2):
        graph = example.Search(model, given, beams, steps).run()
        assert all(torch.equal(a, b) for a, b in zip(eager, graph))
    assert model.status.item() == 0


def test_example_runs(example):
    assert example.main() == 0
