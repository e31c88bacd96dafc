"""examples/tree_decoding.py: the operators together.  At a temperature so low that
sampling is the argmax, drafted trees must emit exactly what decoding one token at
a time does."""
import importlib.util
import os

import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("tree_decoding", os.path.join(ROOT, "examples", "tree_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trees_emit_what_single_steps_do(ex):
    model = ex.Model(seed=3)
    out = []
    for nodes in (1, 8):
        d = ex.Decoder(model, nodes=nodes, temperature=1e-4, seed=nodes)
        seqs = [d.start(range(5, 60)), d.start([9])]
        while min(len(s.tokens) for s in seqs) < 90:
            d.step(seqs)
        d.check()
        out.append([s.tokens[:90] for s in seqs])
        if nodes == 8:
            assert d.accepted > 0, "no drafted token was ever accepted"
    assert out[0] == out[1]


def test_forks_share_and_part(ex):
    """A fork continues as its origin would, and neither disturbs the other."""
    model = ex.Model(seed=4)
    alone = ex.Decoder(model, temperature=1e-4)
    ref = alone.start(range(30))
    while len(ref.tokens) < 80:
        alone.step([ref])
    d = ex.Decoder(model, temperature=1e-4, pages=20)
    a = d.start(range(30))
    while len(a.tokens) < 40:
        d.step([a])
    b = d.fork(a)
    assert b.pages[:len(a.tokens) // 16] == a.pages[:len(a.tokens) // 16]
    while min(len(a.tokens), len(b.tokens)) < 80:
        d.step([a, b])
    d.check()
    assert a.tokens[:80] == ref.tokens[:80] and b.tokens[:80] == ref.tokens[:80]
    d.cache.free(a)
    d.cache.free(b)
    assert d.cache.free_pages == 20


def test_main_runs(ex, capsys):
    ex.main()
    assert "forked:" in capsys.readouterr().out
