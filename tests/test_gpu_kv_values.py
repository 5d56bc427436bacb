"""The paged 8-bit cache and its attention where values are not finite or differ in size by many powers of
two: what a row does not see does not reach it, and what a call does not store leaves no mark."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()


def batch(*args, **kw):
    from test_gpu_kv_attention import Batch
    return Batch(*args, **kw)


def same_cache(a, b):
    for x, y in ((a.k, b.k), (a.v, b.v), (a.ks, b.ks), (a.vs, b.vs)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ---- the append -------------------------------------------------------------------------------------

@pytest.mark.parametrize("new,past,page", [([1], [3], 64), ([1, 1, 1], [3, 3, 70], 16), ([5], [3], 64), ([9, 2], [70, 71], 32),
                                           ([40] * 40, [5] * 40, 16), ([300], [17], 128), ([130, 129], [17, 17], 32)])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, None, False), (128, 64, True), (64, 32, False)])
def test_append_reads_the_rotation_of_its_own_positions(new, past, page, dim, rot, interleaved):
    """Rows of the rotation table that belong to no token of the call may hold anything."""
    a, b = (batch(new, past, 4, 2, dim, page, "int8", "bf16", seed=3, rot=rot, interleaved=interleaved) for _ in range(2))
    used = sorted({p + i for n, p in zip(new, past) for i in range(n)})
    for x in (a, b):
        x.fill_past()
    for t in (b.cos, b.sin):
        kept = t[used].clone()
        t.fill_(float("nan"))
        t[used] = kept
    assert torch.equal(a.append(), b.append())
    same_cache(a, b)


# ---- the attention of prompts ----------------------------------------------------------------------------

def check_with_nan(b, q=None):
    """Every row against the definition: NaN where it sees a value that is, within the bound elsewhere."""
    import kv_util as u
    y = u.values(b.attend(q))
    ref, wabs, xabs = b.reference(q)
    nan = np.isnan(ref)
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(y), nan)
    bound = u.attention_bound(ref, wabs, xabs, b.dtype)
    assert np.all(np.abs(y - ref)[~nan] <= bound[~nan])


PROMPTS = [  # new, past, hq, heads, dim, page
    ([200], [0], 4, 2, 128, 32),
    ([300], [100], 2, 2, 64, 16),                     # one query head a kv head: units of 256 tokens
    ([150, 130], [0, 60], 32, 8, 64, 64),
    ([130, 1, 200], [50, 70, 0], 128, 32, 64, 16),    # more units than CTAs: handed out one by one
    ([70, 1, 90], [3000, 5, 2000], 8, 2, 128, 64),    # a few long units: cut
]


@pytest.mark.parametrize("new,past,hq,heads,dim,page", PROMPTS)
@pytest.mark.parametrize("fmt,dtype", [("int8", "fp16"), ("int8", "bf16"), ("e4m3", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_prompt_rows_before_a_value_that_is_not_finite(new, past, hq, heads, dim, page, fmt, dtype, which):
    """An infinity among a prompt's new values reaches the rows that see its page, and no other."""
    b = batch(new, past, hq, heads, dim, page, fmt, dtype, seed=len(new) + page, rot=0)
    b.fill_past()
    x = b.kn if which == "k" else b.vn
    last = len(new) - 1
    x[int(b.cu_h[last]) + new[last] // 2, heads - 1, 7] = float("inf")
    x[int(b.cu_h[1]) - 1, 0, 1] = float("nan")        # the first prompt's last token
    b.append()
    check_with_nan(b)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16")])
def test_prompt_with_several_pages_that_are_not_finite(fmt, dtype):
    """The first of a head's NaN pages decides; the other heads and sequences keep their own."""
    b = batch([180, 160], [20, 300], 8, 4, 64, 16, fmt, dtype, seed=1)
    b.fill_past()
    b.append()
    for s, head, at in ((0, 1, 9), (0, 1, 4), (0, 3, 12), (1, 0, 25), (1, 2, 20), (1, 2, 28)):
        b.vs[int(b.table_h[s, at]), head] = float("nan")
    b.ks[int(b.table_h[1, 22]), 0] = float("nan")
    check_with_nan(b)


@pytest.mark.parametrize("fmt,dtype", [("int8", "fp16"), ("e4m3", "bf16")])
def test_prompt_ignores_what_no_query_sees(fmt, dtype):
    b = batch([120, 90], [37, 130], 4, 1, 128, 64, fmt, dtype, seed=8)
    b.fill_past()
    b.append()
    y0 = b.attend().clone()
    used = {int(b.table_h[s, at]) for s in range(2) for at in range(-(-(b.past_h[s] + b.new[s]) // 64))}
    for pg in range(b.k.shape[0]):
        if pg not in used:
            b.ks[pg], b.vs[pg] = float("inf"), float("nan")
    for s in range(2):
        held = b.past_h[s] + b.new[s]
        pg, rows = int(b.table_h[s, (held - 1) // 64]), (held - 1) % 64 + 1
        for codes in (b.k, b.v):
            codes.view(torch.uint8)[pg, :, rows:] = 0x7F
    assert torch.equal(b.attend(), y0)


@pytest.mark.parametrize("new,past,hq,heads,dim,page", [([150], [100], 4, 2, 128, 32), ([70, 1, 90], [3000, 5, 2000], 8, 2, 64, 64),
                                                        ([3, 1], [900, 40], 8, 2, 128, 16)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("size", [1e7, 1e8, 1e9, 1e12, 1e30])
def test_scores_beyond_the_steps_of_fp32(new, past, hq, heads, dim, page, fmt, size):
    """Scores so large that neighbouring fp32 values lie apart by more than the weights' range: one position
    takes all the weight, and nothing is NaN."""
    b = batch(new, past, hq, heads, dim, page, fmt, "bf16", seed=5, rot=0)
    b.fill_past()
    b.append()
    q = (b.q.float() * size).to(b.q.dtype)
    y = b.attend(q).float()
    assert not bool(y.isnan().any())
    # an average of the values of its head: none larger than the largest of them, its weights rounded to fp16
    for s in range(len(new)):
        pages = [int(b.table_h[s, at]) for at in range(-(-(past[s] + new[s]) // page))]
        largest = (b.v[pages].float() * b.vs[pages][..., None, None])[:, :, :].nan_to_num(0).abs().amax((0, 2))
        rows = y[int(b.cu_h[s]):int(b.cu_h[s + 1])].view(new[s], heads, hq // heads, dim).abs().amax((0, 2))
        assert bool((rows <= largest * 1.01).all())


@pytest.mark.parametrize("new,past,hq,heads,dim,page", [([150], [100], 4, 2, 128, 32), ([170, 1, 140], [90, 40, 200], 8, 4, 64, 16)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_prompt_rows_before_much_larger_pages(new, past, hq, heads, dim, page, fmt, dtype, which):
    """Later pages of one head are 2^36 times as large as those before them: rows that see only the small
    ones keep all of their bits."""
    import test_gpu_kv_attention as t
    b = batch(new, past, hq, heads, dim, page, fmt, dtype, seed=5, rot=0)
    b.fill_past()
    b.append()
    scales, small, large = (b.ks, -3, 33) if which == "k" else (b.vs, -22, 14) if dtype == "fp16" else (b.vs, 0, 36)
    for s in range(len(new)):
        for at in range(-(-(past[s] + new[s]) // page)):
            behind = at >= (past[s] + new[s] // 2) // page
            scales[int(b.table_h[s, at]), heads - 1] *= 2.0 ** (large if behind else small)
    t.check_attention(b)


@pytest.mark.parametrize("new,past,hq,heads,dim,page", [([1], [0], 2, 1, 128, 16), ([1, 1], [70, 900], 8, 2, 64, 16), ([5, 3], [0, 40], 6, 2, 128, 32),
                                                        ([150], [0], 4, 2, 128, 32), ([60, 1, 70], [3000, 5, 2000], 8, 2, 64, 64)])
@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("value", [float("-inf"), float("inf"), float("nan")])
def test_queries_that_are_not_finite(new, past, hq, heads, dim, page, fmt, dtype, value):
    """A query that is not finite has no softmax: NaN, also where every score is minus infinity; the other
    rows are what they are without it."""
    b = batch(new, past, hq, heads, dim, page, fmt, dtype, seed=2, rot=0)
    b.fill_past()
    b.k.view(torch.uint8)[..., 3] = 0x40              # 64 or 2: channel 3 of every key is above 0
    b.kn[:, :, 3] = 2.0
    b.append()
    q = b.q.clone()
    q[..., 3] = -1.0
    y0 = b.attend(q).clone()
    rows = [(int(b.cu_h[s + 1]) - 1, (3 * s) % hq) for s in range(len(new))]
    for tok, head in rows:
        q[tok, head, 3] = value
    y = b.attend(q)
    bad = torch.zeros(y.shape[:2], dtype=torch.bool, device="cuda")
    for tok, head in rows:
        bad[tok, head] = True
    assert bool(y[bad].isnan().all())
    assert torch.equal(y[~bad], y0[~bad])


def test_rows_that_see_nothing_stay_zero_whatever_their_query():
    b = batch([2, 1], [-2, 5], 4, 2, 64, 16, "int8", "fp16", rot=0)
    b.fill_past()
    b.append()
    q = b.q.clone()
    q[:2] = float("nan")
    y = b.attend(q)
    assert not bool(y[:2].any()) and not bool(y.isnan().any())


@pytest.mark.parametrize("size", [1e30, 1e34, 1e36])
def test_prompt_of_large_queries_and_a_scale_of_zero(size):
    """Scores that count for nothing: every row is the mean of what it sees."""
    import test_gpu_kv_attention as t
    b = batch([130], [40], 4, 2, 64, 16, "e4m3", "bf16", seed=6, rot=0)
    b.fill_past()
    b.append()
    q = torch.randn(b.q.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).clamp(-2, 2)
    t.check_attention(b, q=(q * size).to(b.q.dtype), softmax_scale=0.0)


def roll_back(b, past, new):
    """The same sequences from `past` tokens on, with `new` further ones of b's rows."""
    import gated_deltanet_linear_pre_gb300 as gdn
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    T = int(sum(new))
    rows = torch.cat([torch.arange(int(b.cu_h[s]), int(b.cu_h[s]) + n, device="cuda") for s, n in enumerate(new)])
    gdn.gdn_kv_append(b.cache, cu, T, torch.tensor(past, dtype=torch.int32, device="cuda"), b.table, None, b.kn[rows].contiguous(),
                      b.vn[rows].contiguous(), None, None, False, None)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,page,n_seq,past,new", [
    (128, 16, 1, 5, 9), (64, 32, 3, 20, 3), (128, 64, 2, 40, 40), (64, 128, 1, 30, 90), (128, 128, 2, 3, 120),
    (64, 16, 60, 5, 11), (128, 16, 80, 2, 14), (128, 16, 40, 2, 14), (64, 64, 50, 3, 61)])
def test_rejected_values_that_are_not_finite_do_not_cost_what_was_kept(fmt, dim, page, n_seq, past, new):
    """Drafts of which one is not finite, then an append from in front of it: the page is what it would be
    had that value been 0."""
    heads = 4
    a, b = (batch([new] * n_seq, [past] * n_seq, 4, heads, dim, page, fmt, "bf16", seed=n_seq, rot=0) for _ in range(2))
    kept = new // 2                                   # tokens in front of the one that is not finite
    for x in (a, b):
        x.fill_past()
        for s in range(n_seq):
            row = int(x.cu_h[s]) + kept
            for t, head, c, bad in ((x.kn, 1, 9, float("inf")), (x.vn, 2, 0, float("nan")), (x.vn, 2, 5, float("-inf"))):
                t[row, head, c] = bad if x is b else 0.0
        x.append()
    first = [int(b.table_h[s, (past + kept) // page]) for s in range(n_seq)]
    assert bool(b.ks[first, 1].isnan().all()) and bool(b.vs[first, 2].isnan().all())
    assert not bool(b.ks[first][:, [0, 2, 3]].isnan().any()) and not bool(b.vs[first][:, [0, 1, 3]].isnan().any())
    for codes in ("k", "v"):                          # the finite values of the page are kept beside it
        assert torch.equal(getattr(a, codes).view(torch.uint8), getattr(b, codes).view(torch.uint8))
    # behind the bad value: it stays
    for x in (a, b):
        roll_back(x, [past + kept + 1] * n_seq, [1] * n_seq)
    assert bool(b.ks[first, 1].isnan().all()) and bool(b.vs[first, 2].isnan().all())
    # in front of it: it is gone
    for x in (a, b):
        roll_back(x, [past + kept] * n_seq, [1] * n_seq)
    assert not bool(b.ks[first].isnan().any()) and not bool(b.vs[first].isnan().any())
    same_cache(a, b)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_attend_to_kept_values_after_a_rejected_one(fmt):
    """The kept tokens of a page whose draft was not finite are attended to within their error again."""
    import test_gpu_kv_attention as t
    b = batch([9, 4], [30, 5], 4, 2, 64, 32, fmt, "fp16", seed=4, rot=0)
    b.fill_past()
    b.vn[6, 1, 3] = float("inf")                      # position 36 of the first sequence
    b.kn[11, 0, 3] = float("nan")                     # position 7 of the second
    b.append()
    assert bool(b.attend()[6:9, 2:].isnan().all())
    roll_back(b, [36, 7], [1, 1])
    b.new, b.past_h, b.cu_h, b.T = [1, 1], [36, 7], np.array([0, 1, 2]), 2
    b.cu, b.past = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1, 2], [36, 7]))
    b.q = b.q[:2]
    t.check_attention(b)


def test_a_nan_scale_of_another_hand_stays_until_its_page_begins_afresh():
    """Only the append's own NaN says what the page's scale was."""
    for nan in (0x7FC00000, 0x7FFFFFFF, -1):
        b = batch([3], [4], 2, 2, 64, 16, "int8", "fp16", seed=4, rot=0)
        b.fill_past()
        pg = int(b.table_h[0, 0])
        b.ks.view(torch.int32)[pg, 1] = nan
        b.append()
        assert bool(b.ks[pg, 1].isnan()) and not bool(b.ks[pg, 0].isnan())
        roll_back(b, [1], [2])
        assert bool(b.ks[pg, 1].isnan())
        roll_back(b, [0], [3])
        assert not bool(b.ks[pg].isnan().any())
