"""gdn_adapter_add against the definition in 64 bits.

Tolerances.  A product of two 16-bit values is exact in fp32; a sum of them formed by the tensor core 16 at a time,
in parts that are added up, is off by at most (terms / 16 + 32) steps of 2^-23 of the sum of the terms' sizes.  h
goes on as two pieces: 2^-17 of it in bf16, 2^-21 of its row's largest in fp16.  Then comes a sum of the same kind over
2 * rank terms, and y_out's own rounding: half a step of its type."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

S = 2.0 ** -23
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True, params=["as_chosen", "never_alone"])
def gdn(request, tmp_path_factory):
    """The package, and with a library whose small batches go through the tensor cores' kernels too."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import _native, build
    build.build()
    import gated_deltanet_linear_pre_gb300 as g
    with pytest.MonkeyPatch.context() as m:
        if request.param == "never_alone":
            from selftest_lib import adapter_library
            m.setattr(_native, "_lib", None)
            m.setattr(_native._build, "LIB", adapter_library(str(tmp_path_factory.mktemp("adapter")), "GDN_ADAPTER_SELFTEST_NEVER_ALONE"))
        yield g


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


class Case:
    def __init__(self, lengths, ids, n, rank, d_in, d_out, dt, ranks=None, strided=False, seed=0, up_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dt])
        self.lengths, self.ids, self.dt = lengths, ids, DT[dt]
        self.cu = np.concatenate(([0], np.cumsum(lengths))).astype(int)
        self.T = int(self.cu[-1])
        pad = 16 if strided else 0
        self.x = normal(self.T, d_in + pad)[:, :d_in]
        self.y = normal(self.T, d_out + 3 * pad)[:, pad:pad + d_out]
        self.down, self.up = normal(n, rank, d_in, scale=d_in ** -0.5), normal(n, rank, d_out, scale=up_scale * rank ** -0.5)
        self.ranks = ranks
        if ranks is not None:           # behind an adapter's rank: not read
            for a, r in enumerate(ranks):
                self.down[a, max(r, 0):] = float("nan")
                self.up[a, max(r, 0):] = float("nan")
        self.scales = torch.linspace(-1.5, 2.0, n, device="cuda")

    def run(self, gdn, out=None, stream=None, workspace=None):
        T, (n, rank, d_in) = self.T, self.down.shape
        out = torch.full(self.y.shape, 7.0, dtype=self.dt, device="cuda") if out is None else out
        size = gdn.gdn_adapter_workspace_bytes(len(self.ids), T, rank, d_in)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace[:size]
        gdn.gdn_adapter_add(i32(self.cu), T, i32(self.ids), self.down, self.up, None if self.ranks is None else i32(self.ranks), self.scales,
                            self.x, self.y, out, ws, stream)
        return out

    def check(self, out):
        with np.errstate(invalid="ignore"):
            self._check(out)

    def _check(self, out):
        n, rank, d_in = self.down.shape
        x, y, scales = f64(self.x), f64(self.y), f64(self.scales)
        got, half = f64(out), torch.finfo(self.dt).eps / 2
        tiny = float(torch.finfo(self.dt).smallest_normal) * half
        for s, a in enumerate(self.ids):
            rows = slice(self.cu[s], self.cu[s + 1])
            r = 0 if not 0 <= a < n else rank if self.ranks is None else min(max(self.ranks[a], 0), rank)
            if r == 0:
                assert np.array_equal(got[rows], y[rows]), s
                continue
            if rows.start == rows.stop:
                continue
            down, up = f64(self.down[a, :r]), f64(self.up[a, :r])
            h, size = x[rows] @ down.T, np.abs(x[rows]) @ np.abs(down).T
            dh = (d_in / 16 + 32) * S * size
            dh += 2.0 ** -17 * np.abs(h) if self.dt is torch.bfloat16 else 2.0 ** -21 * np.abs(h).max(1, keepdims=True)
            ref = y[rows] + scales[a] * (h @ up)
            bound = abs(scales[a]) * (dh @ np.abs(up) + (rank / 8 + 32) * S * (np.abs(h) @ np.abs(up))) + 2 * S * np.abs(y[rows])
            off = np.abs(got[rows] - ref)
            limit = bound + half * (np.abs(ref) + bound) + 2 * tiny
            good = (off <= limit) | (~np.isfinite(ref) & ~np.isfinite(got[rows]))
            assert good.all(), (s, a, np.argwhere(~good)[:3].tolist())


MIXED = [1, 0, 17, 64, 5, 130, 16, 1, 33, 63, 0, 65, 48, 2]


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_ranks(gdn, rank, dt):
    rng = np.random.default_rng(rank)
    ids = rng.integers(0, 5, len(MIXED))
    ids[[2, 8]] = -1
    ids[5] = 5
    c = Case(MIXED, ids.tolist(), 5, rank, 520, 712, dt, strided=True)
    c.check(c.run(gdn))


@pytest.mark.parametrize("d_in,d_out", [(8, 8), (24, 64), (64, 72), (72, 1000), (264, 128), (1024, 320), (4104, 56), (2048, 4104)])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("lengths", [[1], [3, 70, 1], [64, 128], [500, 9]])
def test_widths(gdn, d_in, d_out, dt, lengths):
    c = Case(lengths, list(range(len(lengths))), 3, 16, d_in, d_out, dt, seed=d_in)
    c.check(c.run(gdn))


@pytest.mark.parametrize("d_in,d_out,rank", [(65536, 72, 16), (72, 65536, 128), (65528, 65536, 8)])
def test_the_widest(gdn, d_in, d_out, rank):
    c = Case([40, 3, 200], [0, 1, 0], 2, rank, d_in, d_out, "bf16", seed=rank)
    c.check(c.run(gdn))


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 129, 300])
def test_one_sequence(gdn, n):
    for rank in (16, 64):
        c = Case([n], [1], 2, rank, 384, 448, "bf16", seed=n)
        c.check(c.run(gdn))


@pytest.mark.parametrize("rank", [16, 32, 64, 128])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_ranks_of_their_own(gdn, rank, dt):
    ranks = [rank, 1, 0, 5, rank - 3, 8, 13, rank + 9, -4]
    lengths = [3, 40, 5, 1, 70, 16, 2, 17, 4]
    c = Case(lengths, list(range(9)), 9, rank, 264, 328, dt, ranks=ranks)
    c.check(c.run(gdn))


@pytest.mark.parametrize("n_seq,adapters", [(1, 1), (64, 48), (256, 3), (1000, 64)])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_single_tokens(gdn, n_seq, adapters, dt):
    rng = np.random.default_rng(n_seq)
    c = Case([1] * n_seq, rng.integers(-1, adapters, n_seq).tolist(), adapters, 16, 1032, 2056, dt)
    c.check(c.run(gdn))


def test_long_prompts(gdn):
    c = Case([3001, 1, 700, 2500, 4], [2, 1, 2, 0, -1], 3, 64, 1024, 1288, "bf16")
    out = c.run(gdn)
    c.check(out)
    assert torch.equal(out, c.run(gdn))       # the same sums in the same order


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_in_place(gdn, strided, dt):
    c = Case(MIXED, [0, 1, -1, 2, 0, 1, 2, 9, 1, 1, 0, 2, 2, 0], 3, 32, 256, 640, dt, strided=strided)
    want = c.run(gdn)
    whole = c.y._base.clone() if strided else None
    assert torch.equal(c.run(gdn, out=c.y), want)
    if strided:                               # around the slice nothing is written
        whole[:, 16:16 + 640] = want
        assert torch.equal(c.y._base, whole)


def test_a_slice_of_a_packed_projection(gdn):
    """q, k and v of one packed row, each with its own adapters, as the layers' projections leave them."""
    c = Case([40, 1, 9], [1, 0, -1], 2, 16, 256, 384, "fp16")
    packed = torch.randn((c.T, 1024), device="cuda").half()
    before = packed.clone()
    c.y = before[:, 512:896]
    c.run(gdn, out=packed[:, 512:896])
    c.check(packed[:, 512:896])
    packed[:, 512:896] = before[:, 512:896]
    assert torch.equal(packed, before)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_sizes_far_apart(gdn, dt):
    """h far outside fp16's range, and far below it; rows of x that fp16 cannot hold are infinite, and so is what
    comes of them."""
    c = Case([5, 20], [0, 1], 2, 16, 128, 192, dt)
    c.x *= torch.tensor([1.0, 1e4, 1e-4, 3e4, 1.0] * 5, device="cuda")[:, None].to(c.dt)
    c.down[0] *= 100
    c.up[0] = (c.up[0].float() * 2.0 ** -14).to(c.dt)
    c.up[1] *= 0.01
    c.check(c.run(gdn))


@pytest.mark.parametrize("apart", [6, 12, 18, 23])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_small_values_of_h_that_decide(gdn, dt, apart):
    """A token's h whose largest value meets small weights, and its small ones, 2^apart below, large weights: what
    counts is the bits of each value, not those of the largest.

    Tolerances.  h itself is exact here (sums of whole multiples of 2^-apart).  In bf16 its two pieces leave 2^-17 of a
    value; in fp16, scaled to below 2^15, 2^-23 of it or 2^-25, half of the type's least step, which is 2^-39 of the row's
    largest.  The sum over the ranks and the output's rounding as above."""
    c = Case([40, 130, 3], [0, 1, 0], 2, 16, 128, 192, dt, seed=apart)
    c.x.copy_(c.x.float().sign())
    c.down[:, 0] = 64.0
    odd = 65.0 + 2 * torch.arange(15, device="cuda")[:, None]     # 7 bits
    c.down[:, 1:] = (c.down[:, 1:].float().sign() * odd * 2.0 ** -apart).to(c.dt)
    c.up[:, 0] = 2.0 ** -14
    c.up[:, 1:] = (c.up[:, 1:].float().clamp(-1, 1) * 128).to(c.dt)
    c.y.zero_()
    got, eps = f64(c.run(gdn)), torch.finfo(c.dt).eps / 2
    tiny = float(torch.finfo(c.dt).smallest_normal) * eps
    for s, a in enumerate(c.ids):
        rows = slice(c.cu[s], c.cu[s + 1])
        up, scale = f64(c.up[a]), f64(c.scales)[a]
        h = f64(c.x[rows]) @ f64(c.down[a]).T
        dh = np.maximum(2.0 ** -23 * np.abs(h), 2.0 ** -39 * np.abs(h).max(1, keepdims=True)) if dt == "fp16" else 2.0 ** -17 * np.abs(h)
        ref = scale * (h @ up)
        bound = abs(scale) * (dh @ np.abs(up) + (16 / 8 + 32) * S * (np.abs(h) @ np.abs(up)))
        limit = bound + eps * (np.abs(ref) + bound) + 2 * tiny
        off = np.abs(got[rows] - ref)
        assert (off <= limit).all(), (s, float((off / limit).max()))


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_values_that_are_not_finite(gdn, dt):
    c = Case([5, 20, 70], [0, 1, 0], 2, 16, 136, 200, dt)
    want = c.run(gdn)
    c.x[3, 7], c.x[30, 0] = float("nan"), float("inf")
    c.y[10, 5] = float("nan")
    out = c.run(gdn)
    rows = [r for r in range(95) if r not in (3, 30, 10)]
    assert torch.equal(out[rows], want[rows])
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[30]).any()
    assert torch.isnan(out[10, 5]) and int(torch.isnan(out[10]).sum()) == 1
    c = Case([5, 20], [0, 1], 2, 16, 136, 200, dt)
    c.up[1, 3, 9] = float("inf")              # one channel of one adapter
    out = c.run(gdn)
    assert torch.isfinite(out[:5]).all() and not torch.isfinite(out[5:, 9]).any() and int((~torch.isfinite(out)).sum()) == 20


def test_zero_scale_and_zero_weights(gdn):
    c = Case([5, 20], [0, 1], 2, 16, 128, 192, "fp16")
    c.scales[0] = 0
    c.down[1] = 0
    assert torch.equal(c.run(gdn), c.y)


def test_rows_and_weights_past_32_bits(gdn):
    T, d = 140000, 16384                      # y: 2.3e9 elements
    c = Case([3], [0], 1, 8, 64, 64, "bf16")
    y = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda")
    x[-70:] = torch.randn((70, 64), device="cuda").bfloat16()
    n = 20000                                 # up: 2.6e9 elements
    up = torch.zeros((n, 8, d), dtype=torch.bfloat16, device="cuda")
    down = torch.zeros((n, 8, 64), dtype=torch.bfloat16, device="cuda")
    down[n - 1] = torch.randn((8, 64), device="cuda").bfloat16()
    up[n - 1] = torch.randn((8, d), device="cuda").bfloat16()
    scales = torch.ones(n, device="cuda")
    cu = i32([0, T - 70, T])
    ws = torch.empty(gdn.gdn_adapter_workspace_bytes(2, T, 8, 64), dtype=torch.uint8, device="cuda")
    gdn.gdn_adapter_add(cu, T, i32([-1, n - 1]), down, up, None, scales, x, y, y, ws)
    want = (f64(x[-70:]) @ f64(down[-1]).T) @ f64(up[-1])
    # bf16's half step, and far below it the sums of 64 and 8 terms
    assert (np.abs(f64(y[-70:]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-3).all()
    assert int((y[:-70] != 0).any(1).sum()) == 0


@pytest.mark.parametrize("lengths", [[1] * 20, [300, 2, 1]])
def test_another_stream_and_a_graph(gdn, lengths):
    n = len(lengths)
    c = Case(lengths, [i % 3 for i in range(n)], 3, 32, 520, 776, "bf16")
    want = c.run(gdn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run(gdn)
    side.synchronize()
    assert torch.equal(got, want)
    cu, ids, out = i32(c.cu), i32(c.ids), torch.empty_like(c.y)
    ws = torch.empty(gdn.gdn_adapter_workspace_bytes(n, c.T, 32, 520), dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):                        # two graphs on one workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.gdn_adapter_add(cu, c.T, ids, c.down, c.up, None, c.scales, c.x, c.y, out, ws)
        graphs.append(graph)
    for graph, ids_now in zip(graphs, ([2] * n, [-1] + [0] * (n - 1))):
        ids.copy_(i32(ids_now))
        graph.replay()
        c.ids = ids_now
        assert torch.equal(out, c.run(gdn))
        c.check(out)
    # other lengths, as many tokens
    lengths = [c.T - 3 * (n - 1)] + [3] * (n - 1) if c.T > 60 else [0] * 5 + [2] * 5 + [1] * 10
    c.cu = np.concatenate(([0], np.cumsum(lengths))).astype(int)
    cu.copy_(i32(c.cu))
    graphs[0].replay()
    c.check(out)


@pytest.mark.parametrize("rank,d_in,d_out,dt", [(16, 1992, 3080, "fp16"), (32, 520, 5000, "bf16"), (64, 1992, 3080, "bf16"), (128, 1032, 2056, "fp16"),
                                                (72, 2048, 1288, "bf16")])
def test_many_tiles(gdn, rank, d_in, d_out, dt):
    """Prompts and drafts of any length side by side, adapters of any rank and none: ranges that begin and end inside
    tiles, rings that turn many times."""
    rng = np.random.default_rng(rank)
    lengths = [int(x) for x in rng.choice([0, 1, 3, 8, 9, 10, 60, 127, 128, 129, 136, 137, 300, 700], 40)]
    ranks = [rank, 1, rank - 3, 8, rank // 2, 7, 0, rank]
    c = Case(lengths, [int(x) for x in rng.integers(-1, 8, 40)], 8, rank, d_in, d_out, dt, ranks=ranks, strided=True)
    out = c.run(gdn)
    c.check(out)
    assert torch.equal(out, c.run(gdn))
    assert torch.equal(c.run(gdn, out=c.y), out)      # in place


@pytest.mark.parametrize("rank", [24, 40, 72, 104])
def test_low_ranks_among_high_ones(gdn, rank):
    """Prompts cut into ranges by all CTAs, whose adapters use few of the ranks that there is room for."""
    c = Case([4000, 700, 130, 2000], [0, 1, 2, 3], 4, rank, 1024, 2056, "bf16", ranks=[16, 1, 8, 17])
    out = c.run(gdn)
    c.check(out)
    assert torch.equal(out, c.run(gdn))


@pytest.mark.parametrize("lengths", [[1, 3, 2, 1], [300, 2, 1, 5], [200]])
def test_inputs_written_right_before_the_call(gdn, lengths):
    """Every input is new, written by the kernels in front of the call, over buffers that the last call has read."""
    n = len(lengths)
    c = Case(lengths, [i % 3 for i in range(n)], 3, 16, 136, 264, "bf16", ranks=None)
    g = torch.Generator(device="cuda").manual_seed(0)
    cu, ids = i32(c.cu), i32(c.ids)
    ws = torch.empty(gdn.gdn_adapter_workspace_bytes(n, c.T, 16, 136), dtype=torch.uint8, device="cuda")
    news = [[torch.randn(t.shape, generator=g, device="cuda").to(c.dt) for t in (c.x, c.y, c.down, c.up)] for _ in range(40)]
    orders = [torch.randint(-1, 3, (n,), generator=g, device="cuda", dtype=torch.int32) for _ in range(40)]
    out, outs = torch.empty_like(c.y), []
    for new, order in zip(news, orders):
        for t, v in zip((c.x, c.y, c.down, c.up), new):
            t.copy_(v)
        ids.copy_(order)
        gdn.gdn_adapter_add(cu, c.T, ids, c.down, c.up, None, c.scales, c.x, c.y, out, ws)
        outs.append(out.clone())
    for new, order, got in zip(news, orders, outs):
        c.x, c.y, c.down, c.up = new
        c.ids = order.tolist()
        c.check(got)


def test_two_calls_at_once(gdn):
    """Two streams, each with its workspace, several calls each."""
    cases = [Case([500, 3, 260], [0, 1, 1], 2, 64, 1024, 2048, "bf16", seed=1), Case([1] * 200, [i % 2 for i in range(200)], 2, 64, 1024, 2048, "bf16", seed=2),
             Case([130, 900, 1, 1], [1, 0, 1, 0], 2, 64, 1024, 2048, "bf16", seed=3)]
    want = [c.run(gdn).clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                g.append(c.run(gdn))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)


def test_refusals(gdn):
    c = Case([4, 5], [0, 1], 2, 16, 128, 192, "bf16")
    ws = torch.empty(gdn.gdn_adapter_workspace_bytes(2, 9, 16, 128), dtype=torch.uint8, device="cuda")
    good = dict(cu=i32(c.cu), T=9, ids=i32(c.ids), down=c.down, up=c.up, ranks=None, scales=c.scales, x=c.x, y=c.y, out=torch.empty_like(c.y), ws=ws)
    gdn.gdn_adapter_add(*good.values())
    for over in [dict(cu=i32([0, 4])), dict(cu=i32(c.cu).cpu()), dict(ids=i32([0, 1, 2])), dict(ids=torch.zeros(2, device="cuda")), dict(down=c.down.half()),
                 dict(down=c.down[0]), dict(up=c.up[:1]), dict(up=c.up.transpose(1, 2)), dict(ranks=i32([1, 2, 3])), dict(scales=c.scales.double()),
                 dict(x=c.x[:8]), dict(x=c.x[:, :64]), dict(y=c.y.half()), dict(out=c.y[:, :96]), dict(out=c.x), dict(ws=None), dict(ws=ws[:16]),
                 dict(x=c.x.cpu()), dict(out=c.y.t()), dict(down=c.down[:, :12])]:
        with pytest.raises((TypeError, ValueError, gdn.GdnError)):
            gdn.gdn_adapter_add(*(good | over).values())
    none = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_adapter_add(i32([0, 0, 0]), 0, i32([0, 1]), c.down, c.up, None, c.scales, none, none.new_empty((0, 192)), none.new_empty((0, 192)), None)
