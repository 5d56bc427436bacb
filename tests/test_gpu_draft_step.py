"""examples/draft_step.py: the hybrid stack served with drafted tokens.

After some steps the stack's states and caches hold exactly the kept tokens, so the distribution after them
is the one that a fresh stack of the same weights gives after one prefill of the whole text.  Both carry
fp16 activations through 8 layers and an 8-bit cache (whose pages are filled in other pieces, each value
within one code step of the other's), so the logits are compared as distributions, not bit for bit."""
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


def test_served_stack_equals_a_prefill_of_the_kept_tokens(example):
    lines = []
    stack, texts, past = example.serve(n_seq=3, prompt=35, steps=5, drafts=3, seed=3, say=lines.append)
    assert len(lines) == 5
    for s, text in enumerate(texts):
        assert len(text) == int(past[s]) + 1 and all(0 <= t < example.VOCAB for t in text)
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    last = torch.tensor([t[-1] for t in texts], device="cuda")
    served = stack.logits(last, one, past, keep=False)

    fresh = example.HybridStack(3, stack.cos.shape[0], seed=3)
    flat = torch.tensor([t for text in texts for t in text], device="cuda")
    counts = torch.tensor([len(t) for t in texts], dtype=torch.int32, device="cuda")
    whole = fresh.logits(flat, counts, torch.zeros_like(past), keep=False)[counts.cumsum(0) - 1]
    p, q = torch.softmax(served, -1), torch.softmax(whole, -1)
    # total variation: e4m3 rounds a value by up to 2^-4 of it, in both caches at other places, and the logits
    # have a spread of 2; a token or state out of place moves the distribution by order 1
    tv = 0.5 * (p - q).abs().sum(-1)
    assert float(tv.max()) <= 0.1, tv.tolist()


def test_a_step_that_rejects_everything_keeps_one_token(example):
    """Drafts that the target gives no mass: nothing is accepted, and the stack stands one token further."""
    stack = example.HybridStack(2, 64, seed=5)
    past = torch.zeros(2, dtype=torch.int32, device="cuda")
    last = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    drafted = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")   # no such token
    q = torch.full((2, 3, example.VOCAB), 1.0 / example.VOCAB, device="cuda")
    before = [layer.S.clone() for layer in stack.layers if isinstance(layer, example.GdnLayer)]
    drafted_in = drafted.clone()
    # the stack embeds what it is given; give it token 0 where there is no draft
    u = torch.full((2, 4), 0.5, device="cuda")
    orig = stack.embed
    stack.embed = torch.cat((orig, orig[:1]))      # index -1 reads the added row
    accepted, nxt = example.draft_step(stack, last, past, drafted, q, u)
    assert accepted.tolist() == [0, 0] and all(0 <= t < example.VOCAB for t in nxt.tolist())
    assert torch.equal(drafted, drafted_in)
    after = [layer.S for layer in stack.layers if isinstance(layer, example.GdnLayer)]
    assert all(not torch.equal(a, b) for a, b in zip(before, after))
    fresh = example.HybridStack(2, 64, seed=5)
    fresh.logits(last, torch.ones(2, dtype=torch.int32, device="cuda"), past, keep=True)
    for a, b in zip(after, [layer.S for layer in fresh.layers if isinstance(layer, example.GdnLayer)]):
        assert torch.equal(a, b)
