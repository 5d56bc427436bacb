"""gdn_block_norm against the definition in 64 bits.

Tolerances.  With e = 2^-24: a sum of up to 16384 squares is formed by at most 16 multiply-adds a thread and 10
levels of a tree, so it is off by 26 e and its root by 13 e; rsqrtf (2 units), the mean and the weight bring a
norm to 20 e; a sigmoid (expf 2 units, a sum, a division) or SiLU brings u to 32 e, and x' adds its own e.  h
carries x's error through its own value and through its norm, and 20 e of its own.  What is stored in 16 bits
is off by half a step more."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

E = 2.0 ** -24
EPS = 1e-6
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    import gated_deltanet_linear_pre_gb300 as g
    return g


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def unit(x, w):
    return x / np.sqrt((x * x).sum(1, keepdims=True) / x.shape[1] + EPS) * w


def reference(x, y, gate, kind, scale, post, pre):
    """(x', bound of its fp32 error, h, bound), float64."""
    u = np.zeros_like(x)
    if y is not None:
        u = y if post is None else unit(y, post)
        if kind != "none":
            s = 1.0 / (1.0 + np.exp(-gate))
            u = u * {"linear": gate, "sigmoid": s, "silu": gate * s}[kind]
    out = x + scale * u
    ex = 32 * E * np.abs(scale * u) + E * np.abs(out)
    if y is None:
        ex = np.zeros_like(x)
    if pre is None:
        return out, ex, None, None
    h = unit(out, pre)
    rms = np.sqrt((out * out).sum(1, keepdims=True) / x.shape[1] + EPS)
    spread = np.sqrt((ex * ex).sum(1, keepdims=True)) / np.maximum(np.sqrt((out * out).sum(1, keepdims=True)), 1e-30)
    return out, ex, h, ex / rms * np.abs(pre) + np.abs(h) * (spread + 20 * E)


def close(got, ref, bound, what=""):
    half = torch.finfo(got.dtype).eps / 2
    tiny = float(torch.finfo(got.dtype).smallest_normal) * half if got.dtype != torch.float32 else 2.0 ** -149
    off = np.abs(f64(got) - ref)
    limit = bound + half * (np.abs(ref) + bound) + 2 * tiny
    assert (off <= limit).all(), (what, float((off - limit).max()), np.argwhere(off > limit)[:3].tolist())


def inputs(T, width, xt, dt, kind, shared, post, strided, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    pad = 24 if strided else 0
    x = (n(T, width + pad) * 3).to(DT[xt])[:, :width]
    y = n(T, width + 2 * pad).to(DT[dt])[:, pad:pad + width]
    gate = None
    if kind != "none":
        gate = (n(1 if shared else T, width + pad) * 2).to(DT[dt])[:, :width]
    return x, y, gate, (1 + 0.1 * n(width)) if post else None, 1 + 0.1 * n(width)


def call(gdn, x, y, gate, kind, scale, post, pre, stream=None, x_out=True, h=True):
    xo = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") if x_out else None
    ho = torch.full(x.shape, 7.0, dtype=(y if y is not None else x).dtype, device="cuda") if h else None
    gdn.gdn_block_norm(x, y, gate, kind, scale, post, pre if h else None, EPS, xo, ho, stream)
    return xo, ho


def check(gdn, x, y, gate, kind, scale, post, pre):
    xo, ho = call(gdn, x, y, gate, kind, scale, post, pre)
    ref, ex, h, eh = reference(f64(x), f64(y), None if gate is None else f64(gate), kind, scale, None if post is None else f64(post), f64(pre))
    close(xo, ref, ex, "x")
    close(ho, h, eh, "h")


WIDTHS = [8, 64, 248, 256, 264, 504, 512, 520, 1032, 2048, 4096, 5128, 8192, 8200, 12296, 16384]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("xt,dt", [("fp16", "fp16"), ("bf16", "bf16"), ("fp32", "fp16"), ("fp32", "bf16")])
def test_widths(gdn, width, xt, dt):
    check(gdn, *(lambda x, y, g, po, pr: (x, y, g, "sigmoid", 0.7, po, pr))(*inputs(5, width, xt, dt, "sigmoid", False, True, True)))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 157, 700, 2500])
@pytest.mark.parametrize("width", [136, 1000, 4104])
def test_tokens(gdn, T, width):
    x, y, g, po, pr = inputs(T, width, "bf16", "bf16", "silu", False, True, False, seed=T)
    check(gdn, x, y, g, "silu", -1.5, po, pr)


@pytest.mark.parametrize("kind", ["none", "linear", "sigmoid", "silu"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("xt,width,T", [("fp16", 320, 9), ("fp32", 2568, 7), ("fp32", 1536, 1300)])
def test_forms(gdn, kind, shared, post, xt, width, T):
    x, y, g, po, pr = inputs(T, width, xt, "fp16", kind, shared, post, True, seed=3)
    check(gdn, x, y, g, kind, 0.5, po, pr)


@pytest.mark.parametrize("T,width", [(3, 200), (6, 4096), (1500, 2048)])
def test_parts_left_out(gdn, T, width):
    x, y, g, po, pr = inputs(T, width, "fp32", "bf16", "linear", True, True, False)
    xo, ho = call(gdn, x, y, g, "linear", 0.5, po, pr)
    x1, none = call(gdn, x, y, g, "linear", 0.5, po, pr, h=False)
    assert none is None and torch.equal(x1, xo)
    none, h1 = call(gdn, x, y, g, "linear", 0.5, po, pr, x_out=False)
    assert none is None and torch.equal(h1, ho)
    # no block in front: h of x alone
    h2 = torch.empty(x.shape, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_block_norm(x, None, None, "none", 1.0, None, pr, EPS, None, h2)
    _, _, ref, eh = reference(f64(x), None, None, "none", 1.0, None, f64(pr))
    close(h2, ref, eh)


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,width", [(5, 256), (5, 3000), (2000, 2304)])
def test_in_place(gdn, xt, T, width):
    x, y, g, po, pr = inputs(T, width, xt, "bf16", "sigmoid", False, True, False)
    x = x.contiguous()
    want = call(gdn, x, y, g, "sigmoid", 2.0, po, pr)
    h = torch.empty_like(want[1])
    gdn.gdn_block_norm(x, y, g, "sigmoid", 2.0, po, pr, EPS, x, h)
    assert torch.equal(x, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("T,width", [(6, 64), (6, 2056), (1300, 2560)])
def test_rows_do_not_touch_one_another(gdn, T, width):
    """A row with a value that is not finite, a row of zeros, rows of large and of tiny values."""
    x, y, g, po, pr = inputs(T, width, "fp32", "fp16", "linear", False, True, False)
    want = call(gdn, x, y, g, "linear", 1.0, po, pr)
    x[1, 3] = float("nan")
    y[2, 5] = float("inf")
    x[3] = y[3] = 0
    x[4] *= 1e15
    got = call(gdn, x, y, g, "linear", 1.0, po, pr)
    rest = [0] + list(range(5, T))
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(got[1][1]).all() and torch.isnan(got[1][2]).all()
    assert torch.isfinite(got[0][1, 4:]).all() and (got[0][3] == 0).all() and (got[1][3] == 0).all()
    ref, ex, h, eh = reference(f64(x[4:5]), f64(y[4:5]), f64(g[4:5]), "linear", 1.0, f64(po), f64(pr))
    close(got[0][4:5], ref, ex)
    close(got[1][4:5], h, eh)


def test_gates_at_their_ends(gdn):
    x, y, _, _, pr = inputs(4, 64, "fp32", "bf16", "none", False, False, False)
    g = torch.tensor([-3e38, -200.0, -88.0, 0.0, 88.0, 200.0, 3e38, -0.0] * 8, device="cuda").to(torch.bfloat16).expand(4, 64)
    xo, _ = call(gdn, x, y, g, "sigmoid", 1.0, None, pr)
    s = np.array([0, 0, 1 / (1 + np.exp(88.0)), 0.5, 1, 1, 1, 0.5] * 8)
    close(xo, f64(x) + f64(y) * s, 32 * E * np.abs(f64(y) * s) + E * np.abs(f64(x)))
    y[:, 6::8] = 0.5  # silu of the largest value keeps its size
    xo, ho = call(gdn, x, y, g, "silu", 1.0, None, pr)
    assert torch.isfinite(xo).all()


@pytest.mark.parametrize("kind", ["sigmoid", "silu"])
@pytest.mark.parametrize("xt,dt", [("fp16", "fp16"), ("bf16", "bf16"), ("fp32", "fp16"), ("fp32", "bf16")])
def test_the_gates_range(gdn, xt, dt, kind):
    """The gated term alone (x is 0), from gates whose sigmoid a large y makes visible to those that leave y as it is.

    Tolerances, e = 2^-24.  expf is off by 2 units (4 e), the hardware's exponential by 2 + 1.173 |g| units; 1 + exp(-|g|) by e,
    the quotient by 2 units, the products with g, y and scale and the sum by e each: 12 e and the exponential.  An
    exponential below 2^-126 is a multiple of 2^-149, as is its quotient: two of those."""
    big = 60000.0 if dt == "fp16" else 1e38
    ends = [-88.5, -88.0, -87.5, -87.25, -86.0, -40.0, -20.0, -17.0, -9.0, -3.0, -0.5, -1e-3, 0.0, 1e-3, 0.5, 3.0, 9.0, 20.0, 88.0, 200.0, 60000.0, -60000.0]
    g = torch.tensor((ends * 3)[:64], device="cuda").to(DT[dt]).expand(3, 64)
    x = torch.zeros((3, 64), dtype=DT[xt], device="cuda")
    y = torch.full((3, 64), big, dtype=DT[dt], device="cuda")
    y[1], y[2] = 1.0, -big
    if kind == "silu":      # g * y stays in the type's range
        y = torch.where(g > 0.5, torch.full_like(y, 0.5), y)
    xo, _ = call(gdn, x, y, g, kind, 1.0, None, torch.ones(64, device="cuda"))
    gate, u = f64(g), f64(y)
    s = np.where(gate < 0, np.exp(np.minimum(gate, 0)), 1.0) / (1.0 + np.exp(-np.abs(gate)))
    factor = gate if kind == "silu" else 1.0
    ref = u * s * factor
    units = 2.0 if xt == "fp32" else 2.0 + 1.173 * np.abs(gate)
    close(xo, ref, (12 + 2 * units) * E * np.abs(ref) + 2 * 2.0 ** -149 * np.abs(u * factor), kind)


def test_no_tokens(gdn):
    x = torch.empty((0, 128), dtype=torch.float16, device="cuda")
    w = torch.ones(128, device="cuda")
    gdn.gdn_block_norm(x, x.clone(), None, "none", 1.0, None, w, EPS, x.clone(), x.clone())


def test_rows_past_32_bits(gdn):
    T, width = 140000, 16384          # 2.3e9 elements
    x = torch.zeros((T, width), dtype=torch.bfloat16, device="cuda")
    y, h = torch.zeros_like(x), torch.empty_like(x)
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 65536, 131071, 131072, T - 1]
    for r in rows:
        x[r] = torch.randn(width, generator=g, device="cuda")
        y[r] = torch.randn(width, generator=g, device="cuda")
    w = torch.ones(width, device="cuda")
    before = x[rows].clone()
    gdn.gdn_block_norm(x, y, None, "none", 1.0, w, w, EPS, x, h)
    ref, ex, hh, eh = reference(f64(before), f64(y[rows]), None, "none", 1.0, 1.0, np.ones(width))
    close(x[rows], ref, ex)
    close(h[rows], hh, eh)


def test_as_many_rows_as_there_can_be(gdn):
    """2^31 - 1 tokens: four rows a block, whose number is counted past 32 bits on the way."""
    T, width = (1 << 31) - 1, 8
    x = torch.zeros((T, width), dtype=torch.bfloat16, device="cuda")
    h = torch.empty_like(x)
    rows = [0, 3, (1 << 30) + 1, T - 4, T - 1]
    for i, r in enumerate(rows):
        x[r] = torch.arange(width, device="cuda") + i - 3
    w = torch.linspace(0.5, 2.0, width, device="cuda")
    gdn.gdn_block_norm(x, None, None, "none", 1.0, None, w, EPS, None, h)
    at = torch.tensor(rows, device="cuda")
    _, _, ref, eh = reference(f64(x[at]), None, None, "none", 1.0, None, f64(w))
    close(h[at], ref, eh)
    assert not h[T - 1000:T - 4].any() and not h[4:1000].any()


@pytest.mark.parametrize("T,width", [(37, 1016), (3000, 2560)])
def test_another_stream_and_a_graph(gdn, T, width):
    x, y, g, po, pr = inputs(T, width, "bf16", "bf16", "silu", False, True, False)
    want = call(gdn, x, y, g, "silu", 1.0, po, pr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(gdn, x, y, g, "silu", 1.0, po, pr)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    xo, ho = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_block_norm(x, y, g, "silu", 1.0, po, pr, EPS, xo, ho)
    x.mul_(0.5)
    graph.replay()
    want = call(gdn, x, y, g, "silu", 1.0, po, pr)
    torch.cuda.synchronize()
    assert torch.equal(xo, want[0]) and torch.equal(ho, want[1])


def test_refusals(gdn):
    x, y, g, po, pr = inputs(4, 128, "bf16", "bf16", "linear", False, True, False)
    xo, h = torch.empty_like(x), torch.empty_like(x)
    bad = [dict(x=x.cpu()), dict(y=y.half()), dict(y=y[:3]), dict(gate=g[:, :64]), dict(gate=g[:2]), dict(pre=pr[:64]), dict(pre=pr.double()),
           dict(post=po.cpu()), dict(x_out=xo.t()), dict(h=h.float()), dict(h=h[:, ::2]), dict(x=torch.empty((128, 4), device="cuda").t()),
           dict(kind="none"), dict(kind="relu"), dict(eps=0.0), dict(h=xo), dict(x_out=y), dict(x=x[:, 4:124])]
    for over in bad:
        a = dict(x=x, y=y, gate=g, kind="linear", scale=1.0, post=po, pre=pr, eps=EPS, x_out=xo, h=h)
        a.update(over)
        with pytest.raises((TypeError, ValueError, gdn.GdnError)):
            gdn.gdn_block_norm(*a.values())
