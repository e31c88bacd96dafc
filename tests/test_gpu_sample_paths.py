"""Sampled walks on the paths that small cases do not take: shapes of trees that
reject and accept at one node, and batches whose rows are read as the walk meets
them, in every type, alignment and with no drafter scores.  Compared with the
64-bit walk of paged_util where its margin says that rounding cannot turn it."""
import numpy as np
import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from paged_util import sample_reference  # noqa: E402
from test_gpu_verify_sample import Drafted  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _compare(got, target, draft, tokens, parents, u, noise, most_skipped):
    """Every sequence against its 64-bit walk; margins below 1e-3 are not compared."""
    accept, path = (x.cpu().numpy() for x in got)
    B, T = tokens.shape
    skipped = 0
    for b in range(B):
        nodes, token, margin = sample_reference(target[b].double().numpy(), None if draft is None else draft[b].double().numpy(),
                                                tokens[b], parents[b], u[b].astype(np.float64),
                                                noise[b].astype(np.float64), 1.0, T)
        if margin < 1e-3:
            skipped += 1
            continue
        assert accept[b].tolist() == [len(nodes), token], (b, margin)
        assert path[b].tolist() == nodes + [-1] * (T - len(nodes)), b
    assert skipped <= most_skipped * B


@pytest.mark.parametrize("B,V", [(600, 300),    # the statistics of all rows are taken first
                                 (300, 8000)])  # 58 MB: rows are read as the walk meets them
@pytest.mark.parametrize("rejected", [1, 3])
def test_accepted_after_rejections_then_an_only_child_rejected(B, V, rejected):
    """Root -> some rejected children, then an accepted one -> one child, rejected.
    The lists of rejections of the two nodes follow each other at once.  The
    rejected tokens are those by which Q exceeds P most, the accepted one (u = 0)
    that by which P exceeds Q most, so that nearly every walk is of this kind."""
    T = rejected + 3
    r = np.random.default_rng(V + rejected)
    target = torch.from_numpy(r.standard_normal((B, T, V)).astype(np.float32) * 2)
    draft = torch.from_numpy(r.standard_normal((B, T, V)).astype(np.float32) * 2)
    parents = np.zeros((B, T), np.int32)
    parents[:, 0], parents[:, T - 1] = -1, T - 2
    more = torch.softmax(draft, 2) - torch.softmax(target, 2)  # Q - P
    tokens = np.zeros((B, T), np.int32)
    tokens[:, 1:T - 2] = more[:, 0].topk(rejected, 1).indices.numpy()
    tokens[:, T - 2] = more[:, 0].argmin(1).numpy()
    tokens[:, T - 1] = more[:, T - 2].argmax(1).numpy()
    u = np.full((B, T), 0.999, np.float32)
    u[:, T - 2] = 0.0
    noise = r.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)
    args = (target.cuda(), draft.cuda(), _cuda(tokens), _cuda(u), _cuda(noise))
    got = q.verify_sample(*args, parents=_cuda(parents))
    assert (got[1][:, 0] == T - 2).float().mean() > 0.98 and (got[0][:, 0] <= 1).all()
    _compare(got, target, draft, tokens, parents, u, noise, 0.1)
    for _ in range(5):
        again = q.verify_sample(*args, parents=_cuda(parents))
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("B,T,V", [(300, 1, 3000), (100, 4, 3000), (300, 4, 8000)])
@pytest.mark.parametrize("offset", [2.0 ** 20, -2.0 ** 20])
def test_scores_with_a_large_common_offset(B, T, V, offset):
    """A softmax does not depend on an offset.  2^20 is a multiple of the scores' own
    spacing of 1/8 there, so differences of scores are exact in fp32, and so is the
    definition's walk to 64-bit rounding; margins below 1e-3 are not compared."""
    r = np.random.default_rng(V + T)
    target = torch.from_numpy((r.standard_normal((B, T, V)) * 2 + offset).astype(np.float32))
    draft = torch.from_numpy((r.standard_normal((B, T, V)) * 2 + offset).astype(np.float32))
    parents = np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))
    tokens = np.zeros((B, T), np.int32)
    tokens[:, 1:] = target[:, :-1].argmax(2).numpy()  # accepted most often
    u = r.random((B, T)).astype(np.float32)
    noise = r.exponential(size=(B, V)).astype(np.float32) + np.float32(1e-30)
    got = q.verify_sample(target.cuda(), draft.cuda(), _cuda(tokens), _cuda(u), _cuda(noise), parents=_cuda(parents))
    if T > 1:
        assert (got[0][:, 0] == T - 1).float().mean() > 0.25  # nodes without children are reached
    _compare(got, target, draft, tokens, parents, u, noise, 0.1)


@pytest.mark.parametrize("dtype,draft,B,T,V,tree", [
    ("bf16", True, 48, 8, 40000, False),   # 16-byte rows
    ("f16", True, 48, 8, 40008, True),
    ("bf16", True, 48, 8, 40001, True),    # rows of any alignment
    ("f16", True, 48, 8, 40003, False),
    ("f32", True, 24, 8, 40001, True),
    ("bf16", False, 96, 8, 40000, True),   # tokens drafted without probabilities
    ("f16", False, 96, 8, 40001, False),
    ("f32", False, 48, 8, 40004, True),
    ("f32", False, 48, 8, 40001, True),
])
def test_rows_read_as_the_walk_meets_them(dtype, draft, B, T, V, tree):
    """More than 48 MB of scores, parents given: no statistics are taken ahead."""
    d = Drafted(dtype, B, T, V, tree, draft, seed=V + B)
    assert B * (T - 1) * V * d.target.element_size() * (2 if draft else 1) > 48 << 20
    parents = torch.from_numpy(d.parents).cuda()
    d.check(d.call(parents=parents))
    d.check(d.call(ragged=True, parents=parents), ragged=True)


@pytest.mark.parametrize("B", [2, 300])  # statistics first; rows read as the walk meets them
def test_sampling_and_moves_in_a_graph(B):
    """verify_sample, commit and copy_pages captured together and replayed over new
    inputs in the same buffers."""
    T, V, page = 6, 8000, 16
    first, second = (Drafted("f32", B, T, V, True, True, seed=B + i) for i in range(2))
    cache = q.PagedCache(2, 2 * B, page, 1, 1, 64, max_batch=B)
    cache.k_pool.normal_(), cache.v_pool.normal_()
    start = cache.k_pool.clone(), cache.v_pool.clone()
    dev = lambda x: _cuda(np.asarray(x, np.int32))  # noqa: E731
    table, lens, src, dst = dev(np.arange(B)[:, None]), dev([3] * B), dev([0]), dev([2 * B - 1])
    bufs = dict(target=first.target.cuda(), draft=first.draft.cuda(), tokens=_cuda(first.tokens), u=_cuda(first.u),
                noise=_cuda(first.noise), parents=_cuda(first.parents), temperature=_cuda(first.temperature))

    def step():
        accept, path = q.verify_sample(**bufs)
        new = cache.commit(table, lens, path, accept)
        cache.copy_pages(src, dst)
        return accept, path, new

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            captured = step()
    torch.cuda.synchronize()
    for d in (first, second):
        for name, buf in bufs.items():
            x = getattr(d, name)
            buf.copy_(x if isinstance(x, torch.Tensor) else torch.from_numpy(x))
        for pool, old in zip((cache.k_pool, cache.v_pool), start):
            pool.copy_(old)
        want = [x.clone() for x in step()]
        pools = cache.k_pool.clone(), cache.v_pool.clone()
        for pool, old in zip((cache.k_pool, cache.v_pool), start):
            pool.copy_(old)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(captured, want))
        assert torch.equal(cache.k_pool, pools[0]) and torch.equal(cache.v_pool, pools[1])
        d.check(want[:2])
    assert cache.sync_status() == q.QMM_OK
