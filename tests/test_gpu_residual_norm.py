"""residual_norm against its definition in 64 bits."""
import itertools
import math

import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import step_util as U  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def make(M, N, res="f32", y="f32", seed=0, post=False, post_bias=False, bias=False, gate=None, size=1.0, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    a = dict(residual=(mean + size * rnd(M, N)).to(U.TYPES[res]), y=None if y is None else rnd(M, N).to(U.TYPES[y]),
             weight=1 + 0.2 * rnd(N))
    if post:
        a["post_weight"] = 1 + 0.2 * rnd(N)
    if post_bias:
        a["post_bias"] = rnd(N)
    if bias:
        a["bias"] = rnd(N)
    if gate:
        a["gate"] = rnd(N) if gate == "row" else rnd(M, N)
    return a


def check(a, scale=1.0, eps=1e-6, centered=False, dtype=None, **kw):
    (x, ex), h = U.residual_norm(a["residual"], a["y"], a.get("weight"), a.get("bias"), a.get("post_weight"), a.get("post_bias"),
                                 a.get("gate"), scale, eps, centered)
    r, out = q.residual_norm(**a, scale=scale, eps=eps, centered=centered, dtype=dtype, **kw)
    torch.cuda.synchronize()
    if a["y"] is None:
        assert r is a["residual"]
    else:
        U.assert_close(r, x, ex + U.rounding(x, r.dtype), "residual")
    if h is None:
        assert out is None
    else:
        U.assert_close(out, h[0], h[1] + U.rounding(h[0], out.dtype), "norm")
    return r, out


@pytest.mark.parametrize("M,N", [(1, 1), (1, 5120), (8, 5120), (3, 1001), (300, 4), (700, 128), (5, 127), (130, 512), (2, 513), (65, 1024),
                                 (3, 1025), (2, 8191), (2, 8192), (3, 8196), (2, 16384), (1, 16385), (2, 17408), (2, 32768), (1, 32767),
                                 (2000, 600), (1300, 1536)])
@pytest.mark.parametrize("centered", [False, True])
def test_sizes(M, N, centered):
    check(make(M, N, seed=N), centered=centered, dtype=torch.bfloat16)
    check(make(M, N, res="bf16", y="bf16", seed=N, post=True, bias=True, gate="row"), centered=centered, scale=0.3, dtype=torch.float16)


@pytest.mark.parametrize("res,y,out", list(itertools.product(U.TYPES, U.TYPES, U.TYPES)))
def test_types(res, y, out):
    for N in (1040, 77):
        check(make(5, N, res, y, post=True, gate="full", seed=3), dtype=U.TYPES[out])


@pytest.mark.parametrize("post,post_bias,bias,gate,centered", [
    (p, pb, b, g, c) for p, pb, b, g, c in itertools.product([0, 1], [0, 1], [0, 1], [None, "row", "full"], [0, 1]) if p or not pb])
def test_parts(post, post_bias, bias, gate, centered):
    for N in (96, 1280):
        check(make(4, N, post=post, post_bias=post_bias, bias=bias, gate=gate, seed=4), centered=bool(centered), scale=-0.7)


def test_norm_alone_and_sum_alone():
    a = make(6, 2048, res="bf16", y=None)
    check(a, dtype=torch.float32)
    a = make(6, 2048, res="f16", y="f32", post=True)
    a["weight"] = None
    check(a)


@pytest.mark.parametrize("centered", [False, True])
def test_large_means_and_small_rows(centered):
    """A mean a thousand times the spread; rows below eps, and of zeros."""
    check(make(3, 5120, mean=1000.0, seed=5), centered=centered, dtype=torch.float32)
    check(make(3, 640, size=1e-5, y=None, seed=6), centered=centered, dtype=torch.float32)
    a = make(3, 1500, y=None)
    a["residual"].zero_()
    check(a, centered=centered, dtype=torch.float32)
    a = make(2, 1500, y=None)
    a["residual"].mul_(1e15)
    check(a, centered=centered, dtype=torch.float32)


def test_rows_that_are_not_finite():
    """They concern themselves alone."""
    for N in (128, 3000):
        a = make(9, N)
        good = q.residual_norm(**a)
        a["residual"][4, 3] = math.nan
        a["y"][7, N - 1] = math.inf
        r, h = q.residual_norm(**a)
        rest = [i for i in range(9) if i not in (4, 7)]
        assert torch.equal(r[rest], good[0][rest]) and torch.equal(h[rest], good[1][rest])
        assert torch.isnan(h[4]).all() and r[7, N - 1] == math.inf and torch.isnan(r[4, 3])


@pytest.mark.parametrize("N", [512, 515, 5120])
def test_strides_in_place_and_leading_dimensions(N):
    a = make(6, N, res="bf16", post=True, gate="full", seed=7)
    wide = {k: torch.full((2, 3, N + 8), 3.0, dtype=a[k].dtype, device="cuda") for k in ("residual", "y", "gate")}
    for k in wide:
        wide[k][..., :N] = a[k].view(2, 3, N)
    out = torch.full((2, 3, N + 12), 3.0, dtype=torch.bfloat16, device="cuda")
    b = a | {k: w[..., :N] for k, w in wide.items()}
    r, h = check({k: v for k, v in b.items()}, out=out[..., :N], residual_out=wide["residual"][..., :N].clone().contiguous())
    assert (out[..., N:] == 3).all()
    # onto itself
    want = r.clone()
    r2, h2 = q.residual_norm(**b, residual_out=b["residual"])
    assert r2 is b["residual"] and torch.equal(r2, want) and torch.equal(h2, h)
    assert all((w[..., N:] == 3).all() for w in wide.values())


# more rows than are at work at a time: the next ones are fetched ahead
@pytest.mark.parametrize("M,N", [(11000, 7), (6000, 65), (5000, 128), (5000, 100), (5000, 300), (2600, 1001), (700, 3001), (700, 5120),
                                 (200, 16384), (200, 17000), (310, 20001)])
@pytest.mark.parametrize("res,y,out", [("bf16", "f32", "bf16"), ("f32", "bf16", "f16"), ("f16", "f16", "f32")])
def test_many_rows(M, N, res, y, out):
    check(make(M, N, res, y, post=True, gate="full", seed=N), dtype=U.TYPES[out])
    check(make(M, N, res, y, gate="row", bias=True, seed=M), dtype=U.TYPES[out], centered=True)


@pytest.mark.parametrize("M,N", [(5, 777), (700, 3001), (2000, 520)])
@pytest.mark.parametrize("ahead", [1, 2, 5])
def test_many_rows_with_strides(M, N, ahead):
    """Rows that begin anywhere, and results onto the inputs."""
    a = make(M, N, "bf16", "f32", post=True, gate="full", seed=ahead)
    wide = {k: torch.full((M, N + 2 * ahead + 1), 3.0, dtype=a[k].dtype, device="cuda") for k in ("residual", "y", "gate")}
    for k, w in wide.items():
        w[:, ahead:ahead + N] = a[k]
    b = a | {k: w[:, ahead:ahead + N] for k, w in wide.items()}
    r, h = check(b, dtype=torch.float32)
    want, h = r.clone(), h.clone()
    r2, h2 = q.residual_norm(**b, residual_out=b["residual"], out=b["y"], dtype=torch.float32)
    assert r2 is b["residual"] and h2 is b["y"] and torch.equal(r2, want) and torch.equal(h2, h)
    for w in wide.values():
        assert (w[:, :ahead] == 3).all() and (w[:, ahead + N:] == 3).all()


def test_results_onto_inputs():
    for M, N in ((6, 900), (3000, 900)):
        a = make(M, N, "bf16", "bf16", seed=8)
        r, h = q.residual_norm(**a)
        for onto in (dict(residual_out="y"), dict(out="y"), dict(out="residual"), dict(residual_out="residual", out="y"), dict(residual_out="y", out="residual")):
            b = a | dict(residual=a["residual"].clone(), y=a["y"].clone())
            r2, h2 = q.residual_norm(**b, **{k: b[v] for k, v in onto.items()})
            assert torch.equal(r2, r) and torch.equal(h2, h), onto
        b = a | dict(residual=a["residual"].clone())
        x = torch.empty_like(r)
        flat = b["residual"].view(-1)
        for bad in (dict(out=x, residual_out=x), dict(out=b["y"].view(-1).view(torch.float32)[:M // 2 * N].view(-1, N)),
                    dict(out=flat.as_strided((M // 2, N), (2 * N, 1)))):
            c = b if bad["out"].shape[0] == M else b | {k: b[k][:M // 2] for k in ("residual", "y")}
            with pytest.raises(q.QmmError) as e:
                q.residual_norm(**c, **bad)
            assert e.value.code == q.QMM_ERR_INVALID_ARG


def test_rows_do_not_depend_on_their_company():
    for N in (128, 5120, 1001):
        a = make(700, N, seed=8, post=True)
        r, h = q.residual_norm(**a)
        for i in (0, 1, 350, 699):
            one = a | dict(residual=a["residual"][i:i + 1], y=a["y"][i:i + 1])
            r1, h1 = q.residual_norm(**one)
            assert torch.equal(r1[0], r[i]) and torch.equal(h1[0], h[i])


def test_stream_and_graph():
    a = make(5, 640, seed=9)
    want = q.residual_norm(**a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q.residual_norm(**a, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q.residual_norm(**a)
    a["y"].mul_(-2)
    graph.replay()
    want = q.residual_norm(**a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    N = 32768
    M = 2 ** 31 // N + 2
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(N, device="cuda") % 7 + 1
    _, h = q.residual_norm(x, weight=torch.ones(N, device="cuda"))
    _, want = q.residual_norm(x[-1:], weight=torch.ones(N, device="cuda"))
    assert torch.equal(h[-1:], want) and not h[:3].any() and want.any()


def test_refusals():
    a = make(4, 64, post=True, gate="row")

    def refuse(error, **kw):
        with pytest.raises(error):
            q.residual_norm(**(a | kw))

    refuse(ValueError, y=None)
    refuse(ValueError, y=None, post_weight=None, gate=None, weight=None)
    refuse(ValueError, residual=a["residual"].cpu())
    refuse(TypeError, y=a["y"].cpu())
    refuse(ValueError, y=a["y"][:3])
    refuse(TypeError, y=a["y"].double())
    refuse(TypeError, weight=a["weight"].bfloat16())
    refuse(ValueError, weight=a["weight"][:3])
    refuse(ValueError, post_weight=None, post_bias=a["weight"])
    refuse(TypeError, gate=a["gate"].bfloat16())
    refuse(ValueError, gate=a["gate"][:3])
    refuse(TypeError, residual_out=a["residual"].bfloat16())
    refuse(TypeError, out=a["residual"].bfloat16(), dtype=torch.float32)
    refuse(TypeError, dtype=torch.int32)
    refuse(ValueError, y=a["y"].t().contiguous().t())
    refuse(ValueError, weight=None, bias=a["weight"])
    refuse(ValueError, residual=torch.zeros(2, 2, 128, device="cuda")[:, :, ::2], y=torch.zeros(2, 2, 64, device="cuda"))
    for kw in (dict(eps=-1.0), dict(eps=math.nan), dict(scale=math.inf)):
        with pytest.raises(q.QmmError) as e:
            q.residual_norm(**(a | kw))
        assert e.value.code == q.QMM_ERR_INVALID_ARG
    x = torch.zeros(1, 32769, device="cuda")
    with pytest.raises(q.QmmError) as e:
        q.residual_norm(x, weight=x[0].clone())
    assert e.value.code == q.QMM_ERR_SHAPE
    with pytest.raises(q.QmmError):  # rows on top of each other
        q.residual_norm(a["residual"][:1].expand(4, 64).clone(), y=a["y"], weight=a["weight"], out=torch.zeros(1, 64, device="cuda").expand(4, 64))
    r, h = q.residual_norm(a["residual"][:0], a["y"][:0], a["weight"])
    assert r.shape == h.shape == (0, 64)


def test_results_onto_the_gate():
    """Each row onto its own gate's row; a row of gates for all is refused."""
    for M, N in ((6, 900), (3000, 900), (700, 1001), (1, 515)):
        a = make(M, N, "f32", "bf16", post=True, gate="full", seed=10)
        r, h = q.residual_norm(**a, dtype=torch.float32)
        for name, want in (("residual_out", r), ("out", h)):
            b = a | dict(gate=a["gate"].clone())
            got = q.residual_norm(**b, dtype=torch.float32, **{name: b["gate"]})
            assert torch.equal(got[0], r) and torch.equal(got[1], h) and torch.equal(b["gate"], want)
    gates = torch.zeros(6, 900, device="cuda")
    a = make(6, 900, "f32", "bf16", seed=10) | dict(gate=gates[0])
    for kw in (dict(out=gates, dtype=torch.float32), dict(residual_out=gates)):
        with pytest.raises(q.QmmError) as e:
            q.residual_norm(**a, **kw)
        assert e.value.code == q.QMM_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["weight", "bias", "post_weight", "post_bias"])
@pytest.mark.parametrize("onto", ["out", "residual_out"])
@pytest.mark.parametrize("M,N,ld,at,bad", [
    (4, 64, 64, 0, True), (4, 64, 64, 3 * 64, True), (4, 64, 64, 4 * 64, False),  # a row's place; behind the last row
    (1, 64, 64, 0, True), (1, 64, 64, 32, True), (1, 64, 64, 64, False),
    (4, 64, 200, 64, False), (4, 64, 200, 136, False), (4, 64, 200, 63, True), (4, 64, 200, 137, True),  # between rows, and beyond
    (4, 64, 200, 600 + 64, False), (4, 64, 200, 600 + 63, True), (4, 64, 200, -64, False), (4, 64, 200, -63, True)])
def test_outputs_over_weights(name, onto, M, N, ld, at, bad):
    """A weight or bias that a row of an output lies over is refused, one between rows is not."""
    a = make(M, N, post=True, post_bias=True, bias=True, seed=11)
    buffer = torch.zeros(N + M * ld + N, device="cuda")
    vector = buffer[N + at:2 * N + at]
    vector.copy_(a[name])
    b, kw = a | {name: vector}, {onto: buffer.as_strided((M, N), (ld, 1), N), "dtype": torch.float32}
    if bad:
        with pytest.raises(q.QmmError) as e:
            q.residual_norm(**b, **kw)
        assert e.value.code == q.QMM_ERR_INVALID_ARG
    else:
        check(b, **kw)
    assert torch.equal(vector, a[name])
