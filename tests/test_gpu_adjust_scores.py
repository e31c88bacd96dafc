"""adjust_scores and count_tokens against their definitions in 64 bits."""
import math

import numpy as np
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


ALL = ("tokens", "parents", "counts", "prompt", "repetition", "frequency", "presence", "bias", "mask")


class Case:
    """Inputs of one call on the host (numpy) and on the GPU; `have` names the optional ones."""

    def __init__(self, B, T, V, dtype="f32", have=ALL, seed=0, shared_bias=False):
        r = np.random.default_rng(seed)
        self.B, self.T, self.V, self.dtype, self.have = B, T, V, U.TYPES[dtype], have
        self.scores = torch.from_numpy(r.normal(0, 4, (B, T, V)).astype(np.float32)).to(self.dtype).cuda()
        h = self.host = {}
        h["tokens"] = r.integers(0, V, (B, T)).astype(np.int32)
        if T > 3:  # the same token twice on a path
            h["tokens"][:, 3] = h["tokens"][:, 1]
        h["parents"] = np.array([[-1] + [int(r.integers(max(0, i - 3), i)) for i in range(1, T)] for _ in range(B)], np.int32)
        h["counts"] = np.where(r.random((B, V)) < 0.1, r.integers(1, 9, (B, V)), 0).astype(np.int32)
        h["prompt"] = r.random((B, V)) < 0.1
        h["repetition"], h["frequency"], h["presence"] = (r.uniform(a, b, B).astype(np.float32) for a, b in ((0.8, 1.5), (-0.3, 0.6), (-0.4, 0.5)))
        h["bias"] = r.normal(0, 1, V if shared_bias else (B, V)).astype(np.float32)
        h["mask"] = r.random((B, T, V)) < 0.4
        self.args = {k: (U.words(h[k]) if k in ("prompt", "mask") else torch.from_numpy(h[k]).cuda()) for k in have}

    def want(self):
        out, err = np.zeros((self.B, self.T, self.V)), np.zeros((self.B, self.T, self.V))
        x = self.scores.float().cpu().numpy()
        h = {k: v if k in self.have else None for k, v in self.host.items()}
        for b in range(self.B):
            of = lambda k, none=None: none if h[k] is None else h[k][b]  # noqa: E731
            bias = h["bias"] if h["bias"] is None or h["bias"].ndim == 1 else h["bias"][b]
            penal = any(h[k] is not None for k in ("repetition", "frequency", "presence"))
            out[b], err[b] = U.adjust(x[b], of("tokens") if penal else None, of("parents"), of("counts") if penal else None, of("prompt"),
                                      float(of("repetition", 1.0)), float(of("frequency", 0.0)), float(of("presence", 0.0)), bias, of("mask"))
        return torch.from_numpy(out).cuda(), torch.from_numpy(err).cuda()

    def check(self, **kw):
        want, err = self.want()
        out = q.adjust_scores(self.scores, **self.args, **kw)
        torch.cuda.synchronize()
        U.assert_close(out, want, err + U.rounding(want.nan_to_num(neginf=0.0), out.dtype))
        return out


@pytest.mark.parametrize("dtype", U.TYPES)
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (1, 8, 31), (2, 5, 32), (3, 4, 2048), (1, 64, 2049), (2, 16, 4104), (1, 3, 50257), (5, 2, 6000)])
def test_sizes(B, T, V, dtype):
    Case(B, T, V, dtype, seed=V).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,V", [(24, 9, 10001), (24, 9, 10000), (61, 7, 15008), (61, 7, 15009), (300, 2, 2048), (700, 1, 99)])
def test_several_nodes_of_a_range(B, T, V, dtype):
    """Some, all or one of a sequence's nodes walked by the same threads."""
    Case(B, T, V, dtype, seed=V).check()


@pytest.mark.parametrize("V", [999, 2304])
@pytest.mark.parametrize("have", [(), ("mask",), ("bias",), ("bias", "mask"), ("repetition", "prompt"), ("frequency", "counts"),
                                  ("presence", "tokens"), ("presence", "frequency", "tokens", "parents"), ("counts", "prompt", "tokens"),
                                  ("repetition", "tokens", "mask"), ALL])
def test_parts(have, V):
    Case(2, 9, V, "f32", have, seed=1).check()
    Case(2, 9, V, "bf16", have, seed=2, shared_bias=True).check()


@pytest.mark.parametrize("V", [515, 1024])
def test_in_place_strides_and_nodes_past_the_last(V):
    c = Case(3, 6, V, seed=3)
    want, err = c.want()
    wide = torch.full((3, 7, V + 24), 3.0, device="cuda")
    wide[:, :6, 8:8 + V] = c.scores
    x = wide[:, :6, 8:8 + V]
    n = torch.tensor([6, 0, 4], dtype=torch.int32, device="cuda")
    before = wide.clone()
    # every input in wider rows
    args = dict(c.args)
    for k in ("counts", "prompt", "mask", "bias"):
        t = args[k]
        big = torch.zeros(*t.shape[:-1], t.shape[-1] + 8, dtype=t.dtype, device="cuda")
        big[..., :t.shape[-1]] = t
        args[k] = big[..., :t.shape[-1]]
    assert q.adjust_scores(x, **args, n_tokens=n, out=x) is x
    for b, k in enumerate(n.tolist()):
        U.assert_close(x[b, :k], want[b, :k], err[b, :k] + U.rounding(want[b, :k].nan_to_num(neginf=0.0), torch.float32))
        before[b, :k, 8:8 + V] = x[b, :k]
    assert torch.equal(wide, before)


def test_nodes_that_count_for_nothing():
    """Tokens outside the vocabulary; parents that do not come before their node."""
    c = Case(2, 6, 700, have=("tokens", "parents", "presence", "frequency"), seed=4)
    c.host["tokens"][:] = [[5, -1, 700, 6, 6, 2 ** 31 - 1], [1, 2, 3, -2 ** 31, 2, 2]]
    c.host["parents"][:] = [[-1, 0, 1, 3, 3, 9], [-1, 0, 1, -1, 4, -7]]
    for k in ("tokens", "parents"):
        c.args[k] = torch.from_numpy(c.host[k]).cuda()
    # a negative parent ends a path as the root does
    c.check()


def test_values_that_are_not_finite():
    V = 96
    x = torch.zeros(1, 1, V, device="cuda")
    x[0, 0, :6] = torch.tensor([math.nan, math.inf, -math.inf, math.nan, math.inf, -math.inf])
    mask = np.ones((1, 1, V), bool)
    mask[0, 0, 3:6] = False
    out = q.adjust_scores(x, mask=U.words(mask), repetition=torch.tensor([1.5], device="cuda"),
                          prompt=U.words(np.ones((1, V), bool)))[0, 0]
    assert torch.isnan(out[0]) and out[1] == math.inf and out[2] == -math.inf
    assert (out[3:6] == -math.inf).all() and not out[6:].any()
    # nothing allowed
    out = q.adjust_scores(x, mask=U.words(np.zeros((1, 1, V), bool)))
    assert (out == -math.inf).all()


def test_single_nodes():
    c = Case(4, 1, 777, seed=5)
    want, err = c.want()
    a = {k: v for k, v in c.args.items() if k not in ("tokens", "parents")}
    a["mask"] = a["mask"][:, 0]
    out = q.adjust_scores(c.scores[:, 0], **a)
    U.assert_close(out, want[:, 0], (err + U.rounding(want.nan_to_num(neginf=0.0), torch.float32))[:, 0])
    y = c.scores[:, 0].clone()
    assert q.adjust_scores(y, **a, out=y).data_ptr() == y.data_ptr() and torch.equal(y, out)


def test_stream_and_graph():
    c = Case(2, 5, 3000, "bf16", seed=6)
    want = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = q.adjust_scores(c.scores, **c.args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q.adjust_scores(c.scores, **c.args)
    c.args["counts"].zero_()
    c.host["counts"][:] = 0
    c.args["tokens"].add_(1).remainder_(c.V)
    c.host["tokens"] = c.args["tokens"].cpu().numpy()
    graph.replay()
    want, err = c.want()
    U.assert_close(got, want, err + U.rounding(want.nan_to_num(neginf=0.0), got.dtype))


def test_offsets_past_32_bits():
    B, T, V = 3, 64, 1 << 24
    x = torch.ones(B, T, V, dtype=torch.bfloat16, device="cuda")
    counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
    counts[2, V - 1] = 2
    tokens = torch.full((B, T), V - 2, dtype=torch.int32, device="cuda")
    half = torch.full((B,), 0.5, device="cuda")
    q.adjust_scores(x, tokens, counts=counts, frequency=half, out=x)
    assert x[2, 63, V - 1] == 0 and x[2, 63, V - 2] == 1 - 63 * 0.5 and x[2, 63, V - 3] == 1 and x[1, 0, V - 2] == 1


def test_counts():
    r = np.random.default_rng(7)
    B, T, V = 5, 64, 300
    tokens = r.integers(-2, V + 2, (B, T)).astype(np.int32)
    tokens[0, 5:9] = 7  # several of the same token
    accept = np.array([[63, 7], [0, 3], [10, -1], [64, V], [5, V - 1]], np.int32)
    path = np.stack([r.permutation(T) for _ in range(B)]).astype(np.int32)
    path[4, 2] = 99
    path[4, 3] = -1
    want = r.integers(0, 5, (B, V + 4)).astype(np.int32)
    counts = torch.from_numpy(want.copy()).cuda()
    for b in range(B):
        for j in range(min(accept[b, 0], T)):
            if 0 <= path[b, j] < T and 0 <= tokens[b, path[b, j]] < V:
                want[b, tokens[b, path[b, j]]] += 1
        if 0 <= accept[b, 1] < V:
            want[b, accept[b, 1]] += 1
    cuda = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    q.count_tokens(counts[:, :V], cuda(tokens), cuda(path), cuda(accept))
    assert torch.equal(counts.cpu(), torch.from_numpy(want))


def test_with_sampling():
    """Adjusted scores walked by verify_sample, and the counts of what it emitted: a token that a
    grammar forbids is neither accepted nor emitted, one with a large penalty is left after its first use."""
    B, T, V = 2, 4, 64
    scores = torch.zeros(B, T, V, device="cuda")
    scores[..., 5], scores[..., 9] = 40.0, 20.0
    tokens = torch.tensor([[1, 5, 5, 9], [1, 5, 9, 9]], dtype=torch.int32, device="cuda")
    parents = torch.tensor([[-1, 0, 1, 1], [-1, 0, 1, 2]], dtype=torch.int32, device="cuda")
    counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
    mask = np.ones((B, T, V), bool)
    mask[1, :, 5] = False
    frequency = torch.full((B,), 100.0, device="cuda")
    x = q.adjust_scores(scores, tokens, parents, counts=counts, frequency=frequency, mask=U.words(mask))
    accept, path = q.verify_sample(x, None, tokens, torch.full((B, T), 0.5, device="cuda"), torch.ones(B, V, device="cuda"), parents=parents)
    # the first: 5, then 9 (5 was used), then neither; the second: 5 is forbidden, 9 is emitted
    assert accept[0, 0] == 2 and path[0, :2].tolist() == [1, 3] and accept[0, 1] not in (5, 9)
    assert accept[1].tolist() == [0, 9]
    q.count_tokens(counts, tokens, path, accept)
    want = torch.zeros_like(counts)
    want[0, [5, 9, int(accept[0, 1])]] = 1
    want[1, 9] = 1
    assert torch.equal(counts, want)


def test_refusals():
    c = Case(2, 3, 64, seed=8)

    def refuse(error, scores=c.scores, **kw):
        with pytest.raises(error):
            q.adjust_scores(scores, **(c.args | kw))

    refuse(ValueError, c.scores.cpu())
    refuse(ValueError, c.scores[0, 0])
    refuse(TypeError, c.scores.double())
    refuse(ValueError, c.scores.transpose(1, 2).contiguous().transpose(1, 2))
    refuse(ValueError, c.scores[:, 0])
    refuse(ValueError, tokens=c.args["tokens"][:1])
    refuse(TypeError, tokens=c.args["tokens"].long())
    refuse(TypeError, counts=c.args["counts"].cpu())
    refuse(ValueError, counts=c.args["counts"][:, :63])
    refuse(ValueError, prompt=c.args["prompt"][:, :1])
    refuse(ValueError, mask=c.args["mask"][:, :2])
    refuse(TypeError, mask=c.args["mask"].long())
    refuse(TypeError, repetition=c.args["repetition"].double())
    refuse(ValueError, bias=c.args["bias"][:, :5])
    refuse(ValueError, out=torch.empty(2, 3, 65, device="cuda"))
    refuse(TypeError, out=torch.empty(2, 3, 64, dtype=torch.bfloat16, device="cuda"))
    x = torch.zeros(1, 65, 8, device="cuda")
    with pytest.raises(q.QmmError) as e:
        q.adjust_scores(x)
    assert e.value.code == q.QMM_ERR_SHAPE
    y = torch.zeros(2, 2, 8, device="cuda")
    with pytest.raises(q.QmmError) as e:  # onto itself with other strides
        q.adjust_scores(y, out=y.transpose(0, 1))
    assert e.value.code == q.QMM_ERR_INVALID_ARG
    assert q.adjust_scores(c.scores[:0]).shape == (0, 3, 64)
    ok = dict(counts=c.args["counts"], tokens=c.args["tokens"], path=c.args["tokens"], accept=c.args["tokens"][:, :2].contiguous())
    for kw in (dict(path=c.args["tokens"][:, :2]), dict(accept=c.args["tokens"]), dict(counts=c.args["counts"][:1])):
        with pytest.raises(ValueError):
            q.count_tokens(**(ok | kw))
    with pytest.raises(TypeError):
        q.count_tokens(**(ok | dict(counts=c.args["counts"].long())))
