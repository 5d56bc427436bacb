"""GPU parity of gdn_draft_verify: accepted counts and next tokens equal those of the rule written out
sequence by sequence with whole-number weights (tests/kv_util.py)."""
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


def run(p, q, draft, count, u):
    import gated_deltanet_linear_pre_gb300 as gdn
    n = p.shape[0]
    buf = torch.full((2, n + 2), -77, dtype=torch.int32, device="cuda")
    acc, nxt = buf[0, 1:n + 1], buf[1, 1:n + 1]
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    gdn.gdn_draft_verify(dev(p) if isinstance(p, np.ndarray) else p, dev(q) if isinstance(q, np.ndarray) else q, dev(draft),
                         dev(count), dev(u), acc, nxt)
    torch.cuda.synchronize()
    assert bool((buf[:, 0] == -77).all()) and bool((buf[:, -1] == -77).all())
    return acc.cpu().numpy(), nxt.cpu().numpy()


def check(p, q, draft, count, u):
    import kv_util
    acc, nxt = run(p, q, draft, count, u)
    for s in range(p.shape[0]):
        want = kv_util.verify(p[s], q[s], draft[s], draft.shape[1] if count is None else int(count[s]), u[s])
        assert (acc[s], nxt[s]) == want, s
    return acc, nxt


def batch(n, d, vocab, seed, sharp=2.0, apart=0.7):
    rng = np.random.default_rng(seed)
    lq = rng.standard_normal((n, d, vocab)) * sharp
    lp = rng.standard_normal((n, d + 1, vocab)) * apart
    lp[:, :d] += lq
    soft = lambda x: (np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)).astype(np.float32)
    p, q = soft(lp), soft(lq)
    draft = np.zeros((n, d), np.int32)
    for s in range(n):
        for i in range(d):
            draft[s, i] = min(vocab - 1, np.searchsorted(np.cumsum(q[s, i], dtype=np.float64), rng.random()))
    return p, q, draft, rng.random((n, d + 1)).astype(np.float32)


@pytest.mark.parametrize("n,d,vocab", [(1, 4, 1), (3, 1, 2), (9, 5, 37), (5, 7, 1003), (4, 3, 4096), (3, 2, 4097), (2, 40, 515),
                                       (3, 2, 33001), (17, 1, 8192)])
def test_matches_the_rule(n, d, vocab):
    p, q, draft, u = batch(n, d, vocab, seed=n + d + vocab)
    check(p, q, draft, None, u)
    check(p, q, draft, np.random.default_rng(1).integers(-1, d + 2, n).astype(np.int32), u)


def test_all_accepted_and_none():
    p, q, draft, u = batch(6, 4, 300, seed=2)
    p[:, :4] = q                                    # u q < p always (u < 1)
    acc, _ = check(p, q, draft, None, u)
    assert (acc == 4).all()
    for s in range(6):
        for i in range(4):
            p[s, i, draft[s, i]] = 0.0
    acc, nxt = check(p, q, draft, None, u)
    assert (acc == 0).all() and all(nxt[s] != draft[s, 0] for s in range(6))


def test_ends_of_the_unit_interval():
    """u = 0 draws the first token with weight, the largest u below 1 and beyond the last one."""
    p, q, draft, u = batch(4, 1, 600, seed=3)
    count = np.zeros(4, np.int32)
    p[:, 0, :7] = 0.0
    p[:, 0, 590:] = 0.0
    u[:, 1] = [0.0, np.float32(1) - np.float32(2.0 ** -24), 1.0, np.nan]
    import kv_util
    acc, nxt = run(p, q, draft, count, u)
    assert nxt[0] == 7 and nxt[1] == nxt[2] == 589 and nxt[3] == 7
    assert kv_util.verify(p[0], q[0], draft[0], 0, u[0]) == (0, 7)


def test_rows_without_mass():
    p, q, draft, u = batch(5, 2, 100, seed=4)
    u[:, 0] = 1.0
    p[0, 0] = q[0, 0]            # rejected (u = 1), and the residual is 0 everywhere: p itself
    p[1, 0] = 0.0                # no mass at all: -1
    p[2, 0] = np.nan
    p[3, 0, ::2], p[3, 0, 1::2] = -1.0, np.inf      # clamped to 0 and 1
    q[4, 0] = np.nan             # p - q is NaN: p itself
    acc, nxt = check(p, q, draft, None, u)
    assert nxt[1] == -1 and nxt[2] == -1 and 0 <= nxt[0] < 100 and nxt[3] % 2 == 1


def test_drafts_outside_the_vocabulary_are_not_accepted():
    p, q, draft, u = batch(3, 3, 50, seed=5)
    p[:, :3] = q
    draft[0, 1], draft[1, 0], draft[2, 2] = 50, -1, 2 ** 31 - 1
    acc, _ = check(p, q, draft, None, u)
    assert list(acc) == [1, 0, 2]


def test_equal_weights_go_to_the_lowest_index():
    p = np.zeros((3, 1, 5000), np.float32)
    p[:, 0, [10, 2000, 4999]] = 1 / 3
    u = np.array([[0.0], [0.3334], [0.9]], np.float32)
    acc, nxt = run(p, None, None, None, u)
    assert list(acc) == [0, 0, 0] and list(nxt) == [10, 2000, 4999]


def test_strided_rows():
    """Rows of a wider, oddly aligned buffer."""
    p, q, draft, u = batch(4, 2, 777, seed=6)
    base = run(p, q, draft, None, u)
    wide_p, wide_q = np.full((4, 3, 1001), 9, np.float32), np.full((4, 2, 801), 9, np.float32)
    wide_p[..., 3:780], wide_q[..., 1:778] = p, q
    tp, tq = torch.from_numpy(wide_p).cuda()[..., 3:780], torch.from_numpy(wide_q).cuda()[..., 1:778]
    got = run(tp, tq, draft, None, u)
    assert all(np.array_equal(a, b) for a, b in zip(base, got))


def test_largest_vocabulary():
    rng = np.random.default_rng(8)
    V = 1 << 19
    p = rng.random((2, 2, V)).astype(np.float32)
    p /= p.sum(-1, keepdims=True)
    q = np.roll(p[:, :1], 5, -1).copy()
    draft = rng.integers(0, V, (2, 1)).astype(np.int32)
    check(p, q, draft, None, rng.random((2, 2)).astype(np.float32))


def test_kept_tokens_follow_the_target():
    """The distribution of the first kept token is p's: 40000 independent sequences over 6 tokens."""
    rng = np.random.default_rng(9)
    n, V = 40000, 6
    pr = np.array([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], np.float32)
    qr = np.array([0.4, 0.1, 0.1, 0.05, 0.05, 0.3], np.float32)
    draft = rng.choice(V, (n, 1), p=qr / qr.sum()).astype(np.int32)
    p = np.broadcast_to(pr, (n, 2, V)).copy()
    q = np.broadcast_to(qr, (n, 1, V)).copy()
    u = rng.random((n, 2)).astype(np.float32)
    acc, nxt = run(p, q, draft, None, u)
    first = np.where(acc > 0, draft[:, 0], nxt)
    freq = np.bincount(first, minlength=V) / n
    # five standard deviations of a binomial share
    assert np.all(np.abs(freq - pr) <= 5 * np.sqrt(pr * (1 - pr) / n))


def test_refusals():
    import gated_deltanet_linear_pre_gb300 as gdn
    z = lambda *s: torch.zeros(s, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        gdn.gdn_draft_verify(z(2, 3, 8).half(), z(2, 2, 8), i(2, 2), None, z(2, 3), i(2), i(2))
    with pytest.raises(ValueError):
        gdn.gdn_draft_verify(z(2, 3, 8), z(2, 3, 8), i(2, 2), None, z(2, 3), i(2), i(2))
    with pytest.raises(ValueError):
        gdn.gdn_draft_verify(z(2, 3, 8).transpose(0, 1).contiguous().transpose(0, 1), z(2, 2, 8), i(2, 2), None, z(2, 3), i(2), i(2))
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_draft_verify(z(1, 1, (1 << 19) + 1), None, None, None, z(1, 1), i(1), i(1))
    assert e.value.status == 2
    a = i(2)
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_draft_verify(z(2, 3, 8), z(2, 2, 8), i(2, 2), None, z(2, 3), a, a)
    assert e.value.status == 1
    gdn.gdn_draft_verify(z(0, 3, 8), z(0, 2, 8), i(0, 2), None, z(0, 3), i(0), i(0))
