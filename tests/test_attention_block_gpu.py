"""The attention block of examples/attention_block.py on the GPU: prompts in chunks and decoding
against the whole block in 64 bits, and captured steps against the same ones step by step."""

import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import oracle
from tests import attn_util as U

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("attention_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def project(x, weights):
    words, scales, biases = weights
    y = oracle.qmm(bits(x), words.cpu().numpy().view(np.uint32), bits(scales), bits(biases), 4)
    return torch.from_numpy(np.asarray(y, dtype=np.float64))


def whole(block, x):
    """The block's output for one sequence x [n, hidden], its intermediates rounded to bf16 and
    keys and values to the cache's 4 bits, all else in 64 bits."""
    n, hq, hk, D = len(x), block.q_heads, block.cache.kv_heads, block.cache.head_dim
    heads = project(x, block.qkv).bfloat16().view(n, hq + 2 * hk, D)
    pos = torch.arange(n)
    q, k = (U.rope_reference(heads[:, part], w.cpu(), pos, block.inv_freq.cpu(), interleaved=False, eps=1e-6,
                             rope_scale=block.rope_scale)[0].bfloat16()
            for part, w in ((slice(0, hq), block.q_norm), (slice(hq, hq + hk), block.k_norm)))
    k, v = (U.values(*U.quantise(t, block.cache.group_size)) for t in (k, heads[:, hq + hk:]))
    see = pos[None] <= pos[:, None]
    if block.window:
        see &= (pos[None] > pos[:, None] - block.window) | (pos[None] < block.sinks)
    y = torch.empty(n, hq, D, dtype=torch.float64)
    for h in range(hq):
        s = (q[:, h].double() @ k[:, h * hk // hq].T / math.sqrt(D)).masked_fill(~see, -math.inf)
        y[:, h] = torch.softmax(s, -1) @ v[:, h * hk // hq]
    return project(y.bfloat16().view(n, hq * D), block.out)


@pytest.mark.parametrize("chunk", [64, 1000])
@pytest.mark.parametrize("window, sinks", [(0, 0), (50, 3)])
def test_prompts_and_decoding(example, chunk, window, sinks):
    """The code of a key or value next to the border of two codes depends on the last bit of a
    projection's bf16 result, here and in the oracle. At half a step of 2^-8 relative and steps
    of codes of a fifteenth of a group's range (a third of the deviation), under 2 % of the codes
    fall on the other side, a whole step of 0.33 off: 0.33 sqrt(0.02) = 5 % of the values'
    deviation at most. bf16 results add under 1 %."""
    block = example.random_block(512, 8, 2, 64, num_pages=30, page_size=16, theta=1e4, window=window, sinks=sinks)
    g = torch.Generator().manual_seed(chunk)
    lens, count = (130, 1, 77), 5
    prompts = [torch.randn(n, 512, generator=g).bfloat16().cuda() for n in lens]
    steps = torch.randn(count, 3, 512, generator=g).bfloat16().cuda()
    got = example.serve(block, prompts, steps, chunk, 160)
    for b, y in enumerate(got):
        x = torch.cat([prompts[b], steps[:, b]])
        want = whole(block, x)
        assert y.shape == want.shape
        off = (y.double().cpu() - want).norm() / want.norm()
        assert off < 0.06, (b, off)
    assert block.status.item() == 0


def test_captured_steps(example):
    """Replays give what the same calls give one by one, at every length."""
    block = example.random_block(256, 4, 1, 64, num_pages=64, page_size=16)
    prompts = [torch.randn(n, 256, device="cuda").bfloat16() for n in (400, 30)]
    steps = torch.randn(20, 2, 256, device="cuda").bfloat16()
    eager = example.serve(block, prompts, steps, 256, 512, graph=False)
    for _ in range(2):
        graph = example.serve(block, prompts, steps, 256, 512)
        assert all(torch.equal(a, b) for a, b in zip(eager, graph))


def test_example_runs(example):
    assert example.main() == 0
