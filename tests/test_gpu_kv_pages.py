"""gdn_kv_remap, gdn_kv_compact and gdn_kv_copy against plain statements on the host: whole numbers and bits,
which have to be equal; and together with the append and the attention that use the pages."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    import gated_deltanet_linear_pre_gb300 as g
    return g


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


# ---- the definitions ----------------------------------------------------------------------------

def remap_reference(table, page, n_pages, parent, keep, need):
    n_old, width = table.shape
    kept, grow, end = [], [], []
    for p, k, n in zip(parent, keep, need):
        k, n = max(int(k), 0), max(int(n), 0)
        row = [int(x) if 0 <= x < n_pages else -1 for x in table[p][:min(-(-k // page), width)]] if 0 <= p < n_old else []
        kept.append(row)
        grow.append(bool(row) and row[-1] >= 0 and n > k and k < len(row) * page)
        end.append(max(len(row), min(-(-n // page), width)))
    readers = {x for row, g in zip(kept, grow) for x in (row[:-1] if g else row) if x >= 0}
    writer = {}
    for i, row in enumerate(kept):
        if grow[i]:
            writer.setdefault(row[-1], i)
    free = [x for x in range(n_pages) if x not in readers and x not in writer]
    used, taken, missing = n_pages - len(free), 0, 0
    out = np.full((len(kept), width), -1, np.int32)
    src, dst = np.full(len(kept), -1, np.int32), np.full(len(kept), -1, np.int32)
    for i, row in enumerate(kept):
        copied = grow[i] and (row[-1] in readers or writer[row[-1]] != i)
        places = ([len(row) - 1] if copied else []) + list(range(len(row), end[i]))
        out[i, :len(row)] = row
        for at in places:
            new = -1
            if taken < len(free):
                new, taken = free[taken], taken + 1
            else:
                missing += 1
            if copied and at == len(row) - 1 and new >= 0:
                src[i], dst[i] = row[-1], new
            out[i, at] = new
    return out, src, dst, [used + taken, missing]


def compact_reference(table, n_pages):
    ok = (table >= 0) & (table < n_pages)
    used = np.unique(table[ok])
    total = len(used)
    src = used[used >= total]
    dst = np.setdiff1d(np.arange(total), used)
    name = np.arange(n_pages)
    name[src] = dst
    out = np.where(ok, name[np.where(ok, table, 0)], -1)
    pad = np.full(n_pages // 2 - len(src), -1)
    return out, np.concatenate((src, pad)), np.concatenate((dst, pad)), [total, len(src)]


# ---- calls --------------------------------------------------------------------------------------

def padded(table, extra):
    """The table on the device, its rows `extra` entries further apart."""
    full = torch.full((table.shape[0], table.shape[1] + extra), 12345, dtype=torch.int32, device="cuda")
    full[:, :table.shape[1]] = i32(table)
    return full[:, :table.shape[1]]


def remap(gdn, table, page, n_pages, parent, keep, need, extra=0, workspace=None):
    n, width = len(parent), table.shape[1]
    out = padded(np.full((n, width), 99), extra)
    a, b, info = i32([77] * n), i32([77] * n), i32([77, 77])
    ws = workspace if workspace is not None else torch.full((gdn.gdn_kv_remap_workspace_bytes(n_pages, n, width),), 0xA5, dtype=torch.uint8,
                                                            device="cuda")
    gdn.gdn_kv_remap(padded(table, 2 * extra), page, n_pages, i32(parent), i32(keep), i32(need), out, a, b, info, ws)
    return out, a, b, info


def same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w).reshape(tuple(g.shape)))


def check_remap(gdn, table, page, n_pages, parent, keep, need, extra=0):
    got = remap(gdn, table, page, n_pages, parent, keep, need, extra)
    want = remap_reference(table, page, n_pages, parent, keep, need)
    same(got, want)
    out, src, dst, info = want
    # what the copies rely on: no page is copied from and to, none is copied to twice
    assert not set(src[src >= 0]) & set(dst[dst >= 0]) and len(set(dst[dst >= 0])) == (dst >= 0).sum()
    return out, src, dst, info


def random_table(rng, rows, width, n_pages, page, bad=0.0):
    """Rows of any length over a shuffled pool; some share a beginning with an earlier row."""
    held = rng.integers(0, width * page + 1, rows)
    ids = list(rng.permutation(n_pages))
    table = np.full((rows, width), -1, np.int64)
    for r in range(rows):
        n, shared = -(-int(held[r]) // page), 0
        if r and rng.random() < 0.5:
            q = int(rng.integers(0, r))
            shared = min(n, -(-int(held[q]) // page))
            shared = int(rng.integers(0, shared + 1))
            table[r, :shared] = table[q, :shared]
        for j in range(shared, n):
            table[r, j] = ids.pop() if ids else -1
    wild = rng.random(table.shape) < bad
    return np.where(wild, rng.choice([-1, -7, n_pages, 1 << 30], table.shape), table), held


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rows,n,width,n_pages", [(1, 1, 1, 1), (1, 5, 3, 9), (7, 7, 6, 50), (20, 33, 9, 120), (40, 90, 40, 1000), (3, 1200, 5, 300),
                                                  (100, 150, 300, 21000), (9, 17, 4100, 60000), (300, 700, 257, 90001)])
def test_remap(gdn, page, rows, n, width, n_pages):
    rng = np.random.default_rng(rows * 1000 + width + page)
    table, held = random_table(rng, rows, width, n_pages, page, bad=0.03)
    for kind in range(3):
        parent = rng.integers(-1, rows + 1, n) if kind else np.arange(n) % rows
        there = (parent >= 0) & (parent < rows)
        keep = np.where(there, held[np.clip(parent, 0, rows - 1)], 5)
        if kind == 2:
            keep = np.where(rng.random(n) < 0.5, rng.integers(-3, width * page + 40, n), keep)
        need = keep + rng.choice([-9, 0, 0, 1, 3, page, 3 * page + 5], n)
        check_remap(gdn, table, page, n_pages, parent, keep, need, extra=3 * (kind % 2))


def test_remap_by_hand(gdn):
    """Pages of 16; row 0 holds 40 tokens (5, 2, 8), row 1 shares its first two pages and has 7: 33 tokens."""
    table = np.array([[5, 2, 8, -1], [5, 2, 7, -1]])
    # 0 goes on: alone in page 8; 1 goes on twice: the first keeps page 7, the second copies it; a cut to 20 tokens
    # goes on in page 2, which others read; a cut to 32 begins a page; one row is dropped
    out, src, dst, info = check_remap(gdn, table, 16, 12, [0, 1, 1, 0, 1, -1], [40, 33, 33, 20, 32, 9], [41, 34, 64, 21, 33, 0])
    assert out.tolist() == [[5, 2, 8, -1], [5, 2, 7, -1], [5, 2, 0, 1], [5, 3, -1, -1], [5, 2, 4, -1], [-1, -1, -1, -1]]
    assert src.tolist() == [-1, -1, 7, 2, -1, -1] and dst.tolist() == [-1, -1, 0, 3, -1, -1] and info == [8, 0]


@pytest.mark.parametrize("wide", [False, True])
def test_remap_writers_and_readers(gdn, wide):
    """A page's last reader keeps it from its writers, whichever row it is; without one the lowest writer has it."""
    table = np.full((1, 30000 if wide else 4), -1)      # wide: each phase is a launch of its own
    table[0, :2] = [3, 1]
    for reader in (None, 0, 2, 4):
        need = [21] * 5
        if reader is not None:
            need[reader] = 20
        out, src, dst, info = check_remap(gdn, table, 16, 6, [0] * 5, [20] * 5, need)
        keeps = 0 if reader is None else reader
        assert [r for r in range(5) if out[r, 1] == 1] == [keeps]
        assert info == [6, 0] and sorted(dst[dst >= 0]) == [0, 2, 4, 5]


@pytest.mark.parametrize("spare", range(0, 8))
def test_remap_runs_out(gdn, spare):
    """Fewer pages than are wanted: the last to ask get none, and a copy without a page is not listed."""
    table = np.array([[0, 1, -1, -1], [2, 3, -1, -1]])
    out, src, dst, info = check_remap(gdn, table, 16, 4 + spare, [0, 0, 1, 1], [20] * 4, [40, 40, 17, 64])
    assert info == [4 + min(spare, 6), max(6 - spare, 0)]


def test_remap_ends(gdn):
    table = np.array([[0, 1], [2, -1]])
    big = 2 ** 31 - 1
    check_remap(gdn, table, 16, 5, [0, 1, 0, 1], [big, big, -big - 1, 16], [big, 0, big, big])
    check_remap(gdn, table, 128, 5, [big, -big - 1], [5, 5], [300, 1])
    check_remap(gdn, table, 16, 5, [], [], [])
    check_remap(gdn, np.zeros((0, 2)), 16, 5, [0, 1], [5, 5], [30, 30])
    check_remap(gdn, np.zeros((3, 0)), 16, 5, [0, 1], [5, 5], [30, 30])


def test_remap_does_not_depend_on_the_workspace(gdn):
    rng = np.random.default_rng(5)
    for rows, width, n_pages in ((12, 20, 300), (60, 600, 40000)):
        table, held = random_table(rng, rows, width, n_pages, 32)
        args = (table, 32, n_pages, np.arange(2 * rows) // 2, np.repeat(held, 2), np.repeat(held, 2) + 3)
        size = gdn.gdn_kv_remap_workspace_bytes(n_pages, 2 * rows, width)
        want = remap_reference(*args)
        for fill in (0, 255, 127):
            ws = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
            same(remap(gdn, *args, workspace=ws[:size]), want)
            assert (ws[size:] == fill).all()


# ---- compact ------------------------------------------------------------------------------------

def check_compact(gdn, table, n_pages, extra=0, in_place=False):
    a, b = i32([77] * (n_pages // 2)), i32([77] * (n_pages // 2))
    info = i32([77, 77])
    ws = torch.full((gdn.gdn_kv_compact_workspace_bytes(n_pages),), 0xA5, dtype=torch.uint8, device="cuda")
    t = padded(table, extra)
    out = t if in_place else padded(np.full(table.shape, 99), 2 * extra)
    gdn.gdn_kv_compact(t, n_pages, out, a, b, info, ws)
    want = compact_reference(table, n_pages)
    same((out, a, b, info), want)
    return want


@pytest.mark.parametrize("rows,width,n_pages,named", [
    (1, 1, 1, 1), (1, 1, 2, 1), (3, 5, 7, 7), (9, 11, 64, 20), (33, 100, 4096, 1500), (64, 256, 10000, 9999), (100, 300, 40000, 21000),
    (700, 1000, 300007, 250000), (3, 40, 4095, 2), (20, 20, 4097, 300)])
def test_compact(gdn, rows, width, n_pages, named):
    rng = np.random.default_rng(rows + n_pages)
    ids = rng.permutation(n_pages)[:named]
    table = rng.choice(ids, (rows, width))
    table = np.where(rng.random(table.shape) < 0.2, rng.choice([-1, -9, n_pages, 1 << 30], table.shape), table)
    for in_place in (False, True):
        check_compact(gdn, table, n_pages, extra=3, in_place=in_place)


def test_compact_ends(gdn):
    check_compact(gdn, np.full((4, 9), -1), 100)                                        # nothing in use
    check_compact(gdn, np.arange(100).reshape(4, 25), 100)                              # all of it
    out, src, dst, info = check_compact(gdn, np.arange(50, 100).reshape(2, 25), 100)    # the back half
    assert info == [50, 50] and list(src) == list(range(50, 100)) and list(dst) == list(range(50))
    check_compact(gdn, np.arange(50).reshape(2, 25), 100)                               # already at the front
    check_compact(gdn, np.zeros((0, 4), int), 9)
    check_compact(gdn, np.zeros((4, 0), int), 9)
    check_compact(gdn, np.arange(40000, 80000)[None], 80000)


# ---- copy ---------------------------------------------------------------------------------------

def pools(n, n_pages, heads, page, dim, fmt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
    out = []
    for _ in range(n):
        codes = [torch.randint(0, 256, (n_pages, heads, page, dim), generator=g, device="cuda", dtype=torch.uint8).view(dt) for _ in range(2)]
        # any bits, NaNs among them
        scales = [torch.randint(-2 ** 31, 2 ** 31 - 1, (n_pages, heads), generator=g, device="cuda", dtype=torch.int32).view(torch.float32)
                  for _ in range(2)]
        out.append((*codes, *scales))
    return out


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int32)


def check_copy(gdn, layers, a, b):
    n_pages = layers[0][0].shape[0]
    want = [[bits(t).clone() for t in layer] for layer in layers]
    for x, y in zip(a, b):
        if 0 <= x < n_pages and 0 <= y < n_pages:
            for layer, src in zip(want, layers):
                for t, s in zip(layer, src):
                    t[y] = bits(s)[x]
    gdn.gdn_kv_copy(gdn.kv_caches([gdn.kv_cache(*layer) for layer in layers]), i32(a), i32(b))
    for layer, w in zip(layers, want):
        for t, x in zip(layer, w):
            assert torch.equal(bits(t), x)


@pytest.mark.parametrize("heads,page,dim,fmt", [(1, 16, 64, "int8"), (3, 16, 64, "e4m3"), (2, 128, 128, "int8"), (5, 32, 128, "e4m3"),
                                                (16, 64, 128, "int8"), (1024, 16, 64, "e4m3"), (7, 64, 64, "int8")])
@pytest.mark.parametrize("layers", [1, 3])
def test_copy(gdn, heads, page, dim, fmt, layers):
    n = 40 if heads < 1000 else 8
    rng = np.random.default_rng(heads)
    order = rng.permutation(n)
    dst = order[:n // 2]
    src = rng.choice(order[n // 2:], n // 2)
    at = rng.permutation(2 * n)[:n // 2]
    a, b = rng.choice([-1, -5, n, 1 << 30], 2 * n), rng.choice([-1, -5, n, 1 << 30], 2 * n)
    a[at], b[at] = src, dst
    b[at[0]] = -1                       # half a pair
    a[at[1]] = n
    a[at[2]] = b[at[2]]                 # onto itself
    check_copy(gdn, pools(layers, n, heads, page, dim, fmt), a, b)


@pytest.mark.parametrize("n", [0, 1, 2, 31, 255, 256, 1023, 1024, 1025, 2050, 5000])
def test_copy_lists(gdn, n):
    rng = np.random.default_rng(n)
    order = rng.permutation(n + 10)
    a, b = rng.choice(order[n // 2:], n), np.full(n, -1)
    some = rng.permutation(n)[:n // 2]
    b[some] = order[:n // 2]
    check_copy(gdn, pools(2, n + 10, 1, 16, 64, "int8"), a, b)


@pytest.mark.parametrize("layers", [63, 64, 65, 130])
def test_copy_in_many_layers(gdn, layers):
    check_copy(gdn, pools(layers, 9, 2, 16, 64, "e4m3"), [0, 3, 0], [5, 8, 6])


def test_copy_past_32_bits(gdn):
    n = 20000                           # 5.2 GB of keys
    k, v = (torch.zeros((n, 16, 128, 128), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n, 16), device="cuda") for _ in range(2))
    k[n - 1] = 5
    v[17000] = 7
    ks[n - 1], vs[17000] = 2.0, 4.0
    gdn.gdn_kv_copy(gdn.kv_cache(k, v, ks, vs), i32([n - 1, 17000]), i32([3, n - 2]))
    assert (k[3] == 5).all() and (v[n - 2] == 7).all() and (ks[3] == 2).all() and (vs[n - 2] == 4).all()
    assert int((k != 0).flatten(1).any(1).sum()) == 2 and int((v != 0).flatten(1).any(1).sum()) == 2


# ---- together -----------------------------------------------------------------------------------

def test_forked_rows_read_as_rows_of_their_own(gdn):
    """Prompts, each forked three times, the forks going on with tokens of their own, some cut and forked again,
    the pool compacted in between: what attention gives is bit for bit that of sequences that share nothing."""
    heads, hq, dim, page, n_pages, width = 2, 6, 64, 16, 200, 12
    g = torch.Generator(device="cuda").manual_seed(3)

    def pool(n):
        return gdn.kv_cache(*(torch.zeros((n, heads, page, dim), dtype=torch.int8, device="cuda") for _ in range(2)),
                            *(torch.zeros((n, heads), device="cuda") for _ in range(2)))
    layers = [pool(n_pages) for _ in range(2)]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").half()

    def step(cache, table, past, q, k, v, counts):
        cu = i32(np.concatenate(([0], np.cumsum(counts))))
        T = int(sum(counts))
        y, q_out = torch.empty_like(q), torch.empty_like(q)
        gdn.gdn_kv_append(cache, cu, T, i32(past), table, q, k, v, None, None, False, q_out)
        ws = torch.empty(gdn.gdn_kv_attn_workspace_bytes(cache, len(counts), T, hq, table.shape[1]), dtype=torch.uint8, device="cuda")
        gdn.gdn_kv_attn(cache, cu, T, i32(past), table, q_out, dim ** -0.5, y, ws)
        return y

    # a row's history: (tokens in front, (k, v) of each layer) of every piece appended to it
    class Row:
        def __init__(self, pieces=()):
            self.pieces = list(pieces)

    def private(layer, batch, q, k, v, keep, new):
        """The same step over pages of the rows' own, every earlier piece appended to each row by itself."""
        n = len(batch)
        cache, own = pool(n * width), i32(np.arange(n * width).reshape(n, width))
        for r, row in enumerate(batch):
            for past, kv in row.pieces:
                k0, v0 = kv[layer]
                cu = i32([0, k0.shape[0]])
                gdn.gdn_kv_append(cache, cu, k0.shape[0], i32([past]), own[r:r + 1], None, k0, v0, None, None, False, None)
        return step(cache, own, keep, q, k, v, new)

    table = i32(np.full((3, width), -1))
    rows, lengths = [Row() for _ in range(3)], [0, 0, 0]
    plan = [([0, 1, 2], None, [23, 37, 48]),                      # prompts
            ([0, 0, 0, 1, 1, 1, 2, 2, 2], None, [1] * 9),         # each forked
            (list(range(9)), None, [4, 0, 1, 7, 2, 1, 3, 1, 1]),  # drafts, one row idle
            ([8, 0, 3, 3, 4, 6, 7, 2], [30, 24, 41, 20, 37, 48, 49, 25], [2, 1, 1, 5, 1, 1, 1, 1]),  # cut, dropped, forked again
            (list(range(8)), None, [1] * 8)]
    for number, (parent, keep, new) in enumerate(plan):
        keep = [lengths[p] for p in parent] if keep is None else keep
        out = i32(np.full((len(parent), width), 99))
        a, b, info = i32([0] * len(parent)), i32([0] * len(parent)), i32([0, 0])
        ws = torch.empty(gdn.gdn_kv_remap_workspace_bytes(n_pages, len(parent), width), dtype=torch.uint8, device="cuda")
        gdn.gdn_kv_remap(table, page, n_pages, i32(parent), i32(keep), i32([k + x for k, x in zip(keep, new)]), out, a, b, info, ws)
        caches = gdn.kv_caches(layers)
        gdn.gdn_kv_copy(caches, a, b)
        table = out
        if number == 3:
            moves = i32([0] * (n_pages // 2)), i32([0] * (n_pages // 2))
            ws = torch.empty(gdn.gdn_kv_compact_workspace_bytes(n_pages), dtype=torch.uint8, device="cuda")
            gdn.gdn_kv_compact(table, n_pages, table, *moves, info, ws)
            gdn.gdn_kv_copy(caches, *moves)
            assert int(table.max()) < int(info[0])
        assert int(info[1]) == 0 or number == 3
        T = sum(new)
        kv = [(normal(T, heads, dim), normal(T, heads, dim)) for _ in layers]
        q = normal(T, hq, dim)
        before = [Row(rows[p].pieces) for p in parent]
        for layer, cache in enumerate(layers):
            y = step(cache, table, keep, q, *kv[layer], new)
            assert torch.equal(y, private(layer, before, q, *kv[layer], keep, new)), (number, layer)
        at, fresh = 0, []
        for row, k, n in zip(before, keep, new):
            if n:
                row.pieces.append((k, [(x[at:at + n], y[at:at + n]) for x, y in kv]))
            at += n
            fresh.append(row)
        rows, lengths = fresh, [k + n for k, n in zip(keep, new)]


def test_a_captured_step_follows_its_rows(gdn):
    """remap, copy and compact captured once; replayed on other tables and lengths, from two graphs that share a
    workspace, one after the other."""
    rng = np.random.default_rng(1)
    n_pages, width, n = 400, 10, 12
    tables = [random_table(rng, 6, width, n_pages, 16) for _ in range(3)]
    ws = torch.empty(gdn.gdn_kv_remap_workspace_bytes(n_pages, n, width), dtype=torch.uint8, device="cuda")
    t, parent, keep, need = i32(tables[0][0]), i32([0] * n), i32([0] * n), i32([0] * n)
    graphs = []
    for _ in range(2):
        out, a, b, info = i32(np.zeros((n, width))), i32([0] * n), i32([0] * n), i32([0, 0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.gdn_kv_remap(t, 16, n_pages, parent, keep, need, out, a, b, info, ws)
        graphs.append((graph, (out, a, b, info)))
    for table, held in tables:
        for graph, outs in graphs:
            p = rng.integers(0, 6, n)
            k = held[p]
            x = k + rng.integers(0, 30, n)
            t.copy_(i32(table))
            parent.copy_(i32(p)), keep.copy_(i32(k)), need.copy_(i32(x))
            graph.replay()
            torch.cuda.synchronize()
            same(outs, remap_reference(table, 16, n_pages, p, k, x))


def test_another_stream(gdn):
    side = torch.cuda.Stream()
    rng = np.random.default_rng(2)
    table, held = random_table(rng, 50, 700, 40000, 32)
    with torch.cuda.stream(side):
        check_remap(gdn, table, 32, 40000, np.arange(100) // 2, np.repeat(held, 2), np.repeat(held, 2) + 1)
        check_compact(gdn, table, 40000)
        check_copy(gdn, pools(2, 30, 3, 16, 64, "int8"), [3, 4], [7, 9])


def test_refusals(gdn):
    t, n3, two = i32(np.zeros((3, 4))), i32([0] * 3), i32([0, 0])
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    good = dict(table=t, page=16, n_pages=9, parent=n3, keep=n3.clone(), need=n3.clone(), out=t.clone(), a=n3.clone(), b=n3.clone(), info=two, ws=ws)
    gdn.gdn_kv_remap(*good.values())
    for over in [dict(table=t.cpu()), dict(table=t.long()), dict(table=t.t()), dict(out=i32(np.zeros((3, 5)))), dict(parent=i32([0] * 4)),
                 dict(keep=n3.cpu()), dict(need=n3.float()), dict(out=t), dict(page=20), dict(n_pages=0), dict(info=n3), dict(ws=None),
                 dict(ws=ws[:64]), dict(ws=ws.int()), dict(a=None)]:
        with pytest.raises((TypeError, ValueError, gdn.GdnError)):
            gdn.gdn_kv_remap(*(good | over).values())
    four = i32([0] * 4)
    good = dict(table=t, n_pages=9, out=t.clone(), a=four, b=four.clone(), info=two, ws=ws)
    gdn.gdn_kv_compact(*good.values())
    for over in [dict(table=t.cpu()), dict(out=i32(np.zeros((4, 4)))), dict(a=n3), dict(b=four), dict(info=None), dict(ws=ws[:8]), dict(b=four[:3]),
                 dict(out=t[:, :3])]:
        with pytest.raises((TypeError, ValueError, gdn.GdnError)):
            gdn.gdn_kv_compact(*(good | over).values())
    layer = pools(1, 5, 1, 16, 64, "int8")[0]
    cache = gdn.kv_cache(*layer)
    for caches, a, b in [([cache, cache], n3, n3), (None, n3, n3), (cache, n3.cpu(), n3), (cache, n3, i32([0])), (cache, n3.long(), n3),
                         (cache, t, t), ([cache, gdn.kv_cache(*pools(1, 5, 2, 16, 64, "int8")[0])], n3, n3), (cache, layer[2].view(torch.int32)[:, 0], n3)]:
        with pytest.raises((TypeError, ValueError, gdn.GdnError)):
            gdn.gdn_kv_copy(caches, a, b)
    gdn.gdn_kv_copy([], n3, n3)
