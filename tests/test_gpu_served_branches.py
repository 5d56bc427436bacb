"""examples/draft_step.py with branches and adapters: every branch's caches and states hold exactly its own kept
tokens, so the distribution after them is what a fresh stack gives after one prefill of its text (compared as
distributions: fp16 activations through 8 layers and an 8-bit cache, as in test_gpu_draft_step.py)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import draft_step
    return draft_step


@pytest.mark.parametrize("branches,adapters", [(3, 0), (1, 2), (2, 2)])
def test_every_branch_equals_a_prefill_of_its_tokens(example, branches, adapters):
    lines = []
    stack, texts, past = example.serve(n_seq=2, prompt=35, steps=4, drafts=3, seed=3, say=lines.append, branches=branches, adapters=adapters)
    n = 2 * branches
    assert len(lines) == 4 and len(texts) == n == stack.n_seq
    for s, text in enumerate(texts):
        assert len(text) == int(past[s]) + 1
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    last = torch.tensor([t[-1] for t in texts], device="cuda")
    served = stack.logits(last, one, past, keep=False)

    fresh = example.HybridStack(n, stack.cos.shape[0], seed=3, rows=n if branches > 1 else None, adapters=adapters)
    # the same weights: the pages' draw, which comes before the adapters', is of another size
    for a, b in zip(fresh.layers, stack.layers):
        a.adapters = b.adapters
    fresh.ids = getattr(stack, "ids", None)
    flat = torch.tensor([t for text in texts for t in text], device="cuda")
    counts = torch.tensor([len(t) for t in texts], dtype=torch.int32, device="cuda")
    whole = fresh.logits(flat, counts, torch.zeros_like(past), keep=False)[counts.cumsum(0) - 1]
    tv = 0.5 * (torch.softmax(served, -1) - torch.softmax(whole, -1)).abs().sum(-1)
    assert float(tv.max()) <= 0.1, tv.tolist()


def test_branches_share_their_prompts_pages(example):
    stack, texts, past = example.serve(n_seq=2, prompt=100, steps=1, drafts=2, seed=5, say=lambda *_: None, branches=4)
    rows = torch.arange(8, dtype=torch.int32, device="cuda")
    info = stack.remap(rows, past, past)
    table = stack.table.cpu()
    page = example.PAGE
    for prompt, first in ((100, 0), (117, 4)):
        shared = (prompt - 1) // page          # whole pages of all of a prompt but its last token
        assert (table[first:first + 4, :shared] == table[first, :shared]).all()
        own = table[first:first + 4, shared]
        assert len(set(own.tolist())) == 4     # the page that each branch has written into
    named = table[table >= 0].unique().numel()
    assert int(info[0]) == named < int((table >= 0).sum()) and int(info[1]) == 0
