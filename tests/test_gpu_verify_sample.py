"""qmm_verify_sample against its definition in 64 bits, and against the property
that makes it worth having: the emitted tokens are distributed as the target's.

Accepted nodes and tokens are whole numbers decided by comparisons of fp32
values; the definition's smallest relative margin says which walks rounding can
turn.  A probability is off by at most about (|score| + 8) 2^-22 per operation
chain, a renormalised difference P - Q by that over the mass that is left; walks
with a margin below 1e-3 are not compared (about one in a few hundred)."""
import ctypes

import numpy as np
import pytest

import speculative_decode_verification_qmm_gb300 as q
from speculative_decode_verification_qmm_gb300 import _lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from paged_util import TYPES, sample_reference  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


class Drafted:
    def __init__(self, dtype, B, T, V, tree, draft, seed, agree=0.7, wide_tree=False):
        r = np.random.default_rng(seed)
        self.B, self.T, self.V = B, T, V
        target = r.standard_normal((B, T, V)) * 2
        top = r.integers(0, V, (B, T, min(V, 8)))
        np.put_along_axis(target, top, np.take_along_axis(target, top, 2) + 6 + r.standard_normal(top.shape), 2)
        noisy = target + r.standard_normal((B, T, V)) * agree
        self.parents = np.full((B, T), -1, np.int32)
        self.tokens = r.integers(0, V, (B, T)).astype(np.int32)
        for b in range(B):
            for i in range(1, T):
                self.parents[b, i] = r.integers(0, 2) if wide_tree and i < 9 else \
                    (r.integers(max(0, i - 4), i) if tree else i - 1)
                if self.parents[b, i] >= i:
                    self.parents[b, i] = 0
            race = noisy[b] + r.gumbel(size=(T, V))
            order = np.argsort(-race, 1)
            used = [0] * T
            for i in range(1, T):
                par = self.parents[b, i]
                if used[par] < V:
                    self.tokens[b, i] = order[par, used[par]]
                used[par] += 1
        self.target = torch.from_numpy(target).to(TYPES[dtype])
        self.draft = torch.from_numpy(noisy).to(TYPES[dtype]) if draft else None
        self.u = r.random((B, T)).astype(np.float32)
        self.noise = r.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)
        self.temperature = (0.6 + 0.8 * r.random(B)).astype(np.float32)
        self.n_tokens = r.integers(1, T + 1, B).astype(np.int32)
        self.tree = tree

    def call(self, ragged=False, **kw):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        args = dict(target=self.target.cuda(), draft=self.draft.cuda() if self.draft is not None else None,
                    tokens=dev(self.tokens), u=dev(self.u), noise=dev(self.noise),
                    parents=dev(self.parents) if self.tree else None, temperature=dev(self.temperature),
                    n_tokens=dev(self.n_tokens) if ragged else None)
        return q.verify_sample(**{**args, **kw})

    def check(self, got, ragged=False, most_skipped=0.1):
        accept, path = (x.cpu().numpy() for x in got)
        skipped = 0
        for b in range(self.B):
            n = int(self.n_tokens[b]) if ragged else self.T
            nodes, token, margin = sample_reference(
                self.target[b].double().numpy(), self.draft[b].double().numpy() if self.draft is not None else None,
                self.tokens[b], self.parents[b], self.u[b].astype(np.float64), self.noise[b].astype(np.float64),
                float(self.temperature[b]), n)
            if margin < 1e-3:
                skipped += 1
                continue
            assert accept[b].tolist() == [len(nodes), token], (b, margin)
            assert path[b].tolist() == nodes + [-1] * (self.T - len(nodes)), b
        assert skipped <= max(2, most_skipped * self.B)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,T,V,tree", [
    (3, 1, 40, False),       # nothing drafted
    (5, 2, 1, False),        # one token in the vocabulary
    (7, 5, 33, True),        # fewer entries than threads, odd
    (4, 8, 1000, False),     # whole groups of 16 bytes
    (6, 16, 4099, True),     # odd rows: single entries
    (2, 64, 20008, True),
    (70, 4, 900, True),      # many sequences: small clusters
])
def test_walks(dtype, draft, B, T, V, tree):
    d = Drafted(dtype, B, T, V, tree, draft, seed=B * T + V)
    d.check(d.call())
    d.check(d.call(ragged=True), ragged=True)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B", [2, 40])
def test_many_siblings(draft, B):
    """Eight children to try at the root and its first child, from a drafter that is
    mostly wrong: several rejections in a row at one node."""
    d = Drafted("f32", B, 20, 5000, True, draft, seed=3, agree=4.0, wide_tree=True)
    d.check(d.call())


@pytest.mark.parametrize("T,V", [(8, 151936), (12, 50257)])
def test_large_vocabulary(T, V):
    d = Drafted("f32", 2, T, V, True, True, seed=T)
    d.check(d.call())


def test_chains_with_and_without_parents_agree():
    """90 MB of scores: a chain without parents has its statistics taken first, one
    whose parents are given is read as the walk meets its rows."""
    d = Drafted("f32", 40, 8, 40000, False, True, seed=12)
    first = [x.cpu() for x in d.call()]
    d.check(first)
    walked = [x.cpu() for x in d.call(parents=torch.from_numpy(d.parents).cuda())]
    assert torch.equal(first[0], walked[0]) and torch.equal(first[1], walked[1])


def test_read_ahead_and_walked_rows_agree():
    """The same sequences alone (statistics of all rows taken first) and in a batch
    large enough for rows to be read as the walk meets them."""
    d = Drafted("f32", 300, 6, 6000, True, True, seed=8)
    whole = [x.cpu() for x in d.call()]
    d.check(whole)
    for b in (0, 7, 150):
        one = q.verify_sample(d.target[b:b + 1].cuda(), d.draft[b:b + 1].cuda(),
                              *(torch.from_numpy(x[b:b + 1].copy()).cuda() for x in (d.tokens, d.u, d.noise)),
                              parents=torch.from_numpy(d.parents[b:b + 1].copy()).cuda(),
                              temperature=torch.from_numpy(d.temperature[b:b + 1].copy()).cuda())
        assert torch.equal(one[0].cpu(), whole[0][b:b + 1]) and torch.equal(one[1].cpu(), whole[1][b:b + 1])


def test_strided_scores_without_a_last_draft_row():
    """Rows of a wider buffer, T - 1 draft rows, columns past V that are never read."""
    d = Drafted("f32", 4, 6, 1000, True, True, seed=9)
    wide = torch.full((4, 7, 1100), float("nan"), device="cuda")
    wide[:, :6, :1000] = d.target.cuda()
    dwide = torch.full((4, 5, 1003), float("nan"), device="cuda")
    dwide[:, :, 1:1001] = d.draft[:, :5].cuda()
    d.check(d.call(target=wide[:, :6, :1000], draft=dwide[:, :, 1:1001]))


@pytest.mark.parametrize("V", [1000, 1001])
def test_masked_vocabulary(V):
    """Scores of -inf and of the type's lowest value are never emitted or accepted."""
    d = Drafted("f32", 30, 5, V, True, True, seed=10)
    gone = torch.zeros(V, dtype=torch.bool)
    gone[::3] = True
    low = torch.zeros(V, dtype=torch.bool)
    low[1::3] = True
    for x in (d.target, d.draft):
        x[:, :, gone] = -float("inf")
    d.target[:, :, low] = torch.finfo(torch.float32).min
    d.check(d.call(), most_skipped=0.3)
    accept, path = (x.cpu().numpy() for x in d.call())
    for b in range(d.B):
        assert accept[b, 1] % 3 == 2
        assert all(d.tokens[b, i] % 3 == 2 for i in path[b, :accept[b, 0]])


def test_large_scores_and_small_temperature():
    """Scores of hundreds at a temperature of 0.05: exponents in the thousands."""
    d = Drafted("f32", 10, 5, 3000, False, True, seed=11)
    d.target *= 40
    d.draft *= 40
    d.temperature[:] = 0.05
    d.check(d.call(), most_skipped=0.5)


def test_equal_scores_tie_to_the_lowest_index():
    T, V = 3, 70
    z = torch.zeros(1, T, V, device="cuda")
    one = torch.ones(1, V, device="cuda")
    tok = torch.tensor([[5, 6, 7]], dtype=torch.int32, device="cuda")
    accept, path = q.verify_sample(z, z, tok, torch.full((1, T), 0.999, device="cuda"), one)
    assert accept.tolist() == [[2, 0]] and path.tolist() == [[1, 2, -1]]
    # nothing of P is left where both are the same and a child is refused
    accept, path = q.verify_sample(z, z, tok, torch.full((1, T), 1.5, device="cuda"), one)
    assert accept.tolist() == [[0, 0]] and path.tolist() == [[-1, -1, -1]]


def test_bad_inputs_stay_in_range():
    """Tokens and parents out of range are nodes that do not exist; NaN scores, zero
    noise and temperatures that are none give some token of the vocabulary."""
    d = Drafted("f32", 6, 8, 500, True, True, seed=12)
    clean = d.call()
    bad = Drafted("f32", 6, 8, 500, True, True, seed=12)
    d.tokens[:, 7], d.parents[:, 7] = 500, 3
    bad.tokens[:, 7], bad.parents[:, 7] = 0, 2 ** 30
    got, want = d.call(), bad.call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    n = torch.tensor([9, -1, 0, 8, 100, 1], dtype=torch.int32, device="cuda")
    accept, path = d.call(n_tokens=n)
    assert (accept[1:3, 0] == 0).all() and (accept[:, 1] >= 0).all() and (accept[:, 1] < 500).all()
    for kw in (dict(target=torch.full((6, 8, 500), float("nan"), device="cuda")),
               dict(target=torch.full((6, 8, 500), -float("inf"), device="cuda")),
               dict(noise=torch.zeros(6, 500, device="cuda")),
               dict(temperature=torch.tensor([0.0, -1.0, float("nan"), float("inf"), 1e-40, 1.0], device="cuda"))):
        accept, path = d.call(**kw)
        assert ((accept[:, 1] >= 0) & (accept[:, 1] < 500)).all()
        assert ((accept[:, 0] >= 0) & (accept[:, 0] < 8)).all()
    assert clean[0].shape == (6, 2)


def test_first_token_is_distributed_as_the_target():
    """200,000 one-step trees of two siblings and a chain over six tokens: the first
    emitted token's frequencies are the target's probabilities.  A frequency's
    standard deviation is at most 0.5 / sqrt(200000) = 0.0011; five of them."""
    B, T, V = 50000, 4, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    target = torch.tensor([1.0, 0.2, -1.0, 0.7, 0.0, -0.3], device="cuda").repeat(B, T, 1)
    target[:, 1:] += torch.randn(T - 1, V, generator=g, device="cuda")
    draft = torch.tensor([-0.5, 1.2, 0.3, 0.0, 0.1, -2.0], device="cuda").repeat(B, T, 1)
    parents = torch.tensor([-1, 0, 0, 1], dtype=torch.int32, device="cuda").repeat(B, 1)
    seen = torch.zeros(V, device="cuda")
    for _ in range(4):
        def rnd(*s):
            return torch.rand(*s, generator=g, device="cuda")
        race = draft[:, 0] - torch.log(-torch.log(rnd(B, V)))
        two = race.topk(2, 1).indices.to(torch.int32)  # drawn without replacement
        third = (draft[:, 1] - torch.log(-torch.log(rnd(B, V)))).argmax(1).to(torch.int32)
        tokens = torch.stack([torch.zeros_like(third), two[:, 0], two[:, 1], third], 1).contiguous()
        noise = torch.empty(B, V, device="cuda").exponential_(generator=g)
        accept, path = q.verify_sample(target, draft, tokens, rnd(B, T), noise, parents=parents)
        first = torch.where(accept[:, 0] > 0, tokens.gather(1, path[:, :1].long().clamp(min=0))[:, 0], accept[:, 1])
        seen += torch.bincount(first.long(), minlength=V)
    want = torch.softmax(target[0, 0], 0)
    assert ((seen / seen.sum() - want).abs() < 0.0056).all()


def test_repeats_and_side_stream():
    d = Drafted("bf16", 5, 9, 7000, True, True, seed=13)
    first = d.call()
    for _ in range(3):
        again = d.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = d.call(stream=s)
    s.synchronize()
    assert torch.equal(first[0], other[0]) and torch.equal(first[1], other[1])


def test_refusals():
    d = Drafted("f32", 2, 3, 100, True, True, seed=14)
    for kw in (dict(draft=d.draft.half().cuda()), dict(tokens=torch.zeros(2, 3, dtype=torch.int64, device="cuda")),
               dict(u=torch.zeros(2, 3)), dict(noise=torch.zeros(2, 100, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            d.call(**kw)
    for kw in (dict(draft=d.draft[:, :1].cuda()), dict(noise=torch.zeros(2, 99, device="cuda")),
               dict(temperature=torch.ones(3, device="cuda")), dict(target=d.target),
               dict(noise=torch.zeros(100, 2, device="cuda").t()),
               dict(target=torch.zeros(2, 100, 3, device="cuda").transpose(1, 2))):
        with pytest.raises(ValueError):
            d.call(**kw)
    with pytest.raises(q.QmmError) as e:
        q.verify_sample(torch.zeros(1, 65, 8, device="cuda"), None, torch.zeros(1, 65, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, 65, device="cuda"), torch.ones(1, 8, device="cuda"))
    assert e.value.code == q.QMM_ERR_SHAPE
    L = q.load()
    a = _lib.qmm_sample_args()
    assert L.qmm_verify_sample(None, None) == q.QMM_ERR_INVALID_ARG
    assert L.qmm_verify_sample(ctypes.byref(a), None) == q.QMM_ERR_INVALID_ARG
    n = ctypes.c_int64(-1)
    for B, T, V in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (65536, 1, 1), (1, 65, 1), (1, 1, (1 << 24) + 1)):
        assert L.qmm_verify_sample_workspace(B, T, V, ctypes.byref(n)) == q.QMM_ERR_SHAPE
    assert L.qmm_verify_sample_workspace(1, 1, 1, None) == q.QMM_ERR_INVALID_ARG
    t = torch.zeros(2, 3, 100, device="cuda")
    ints = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(q.QmmError) as e:  # workspace too small
        q.qmm_verify_sample(t, t, ints, torch.zeros(2, 3, device="cuda"), torch.ones(2, 100, device="cuda"),
                            torch.zeros(2, 2, dtype=torch.int32, device="cuda"), ints.clone(),
                            torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == q.QMM_ERR_INVALID_ARG
