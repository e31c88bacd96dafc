"""examples/tree_decoding.py with penalties: a drafted node is penalised as if the nodes
before it had been emitted one at a time."""
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


def test_trees_with_penalties_emit_what_single_steps_would(ex):
    """Every emitted token is the best one after the tokens before it, up to roundings.

    A score is h . w with |h| = sqrt(HIDDEN); h is rounded to bf16, each entry by at
    most 2^-8 of it, so by the inequality of Cauchy and Schwarz two evaluations differ
    by at most 2 2^-8 sqrt(HIDDEN) |w| for it, and by no more again for what the
    layers round, which add a small part to h.  The penalties take more than that off
    a score of 12."""
    model = ex.Model(seed=5)
    repetition, presence = 1.5, 1.0
    d = ex.Decoder(model, temperature=1e-4, repetition=repetition, presence=presence)
    seqs = [d.start(range(5, 60)), d.start([9])]
    while min(len(s.tokens) for s in seqs) < 80:
        d.step(seqs)
    d.check()
    assert d.accepted > 0
    tol = 4 * 2.0 ** -8 * ex.HIDDEN ** 0.5 * model.head.dequantize().norm(dim=1).max().item()
    penalised = 0
    for s, n in zip(seqs, (55, 1)):
        emitted = torch.tensor(s.tokens[n:])
        assert torch.equal(s.counts.cpu(), torch.bincount(emitted, minlength=ex.VOCAB).int())
        single = ex.Decoder(model, nodes=1)
        for i in range(n, 80):
            one = single.start(s.tokens[:i])
            single.cache.reserve([one], 1)
            last = torch.tensor([[s.tokens[i - 1]]], dtype=torch.int32, device="cuda")
            raw = model.forward(single.cache, last, torch.zeros_like(last), *single.cache.tables([one]), None)[0, 0].double().cpu()
            single.cache.free(one)
            seen = torch.zeros(ex.VOCAB, dtype=torch.bool)
            seen[s.tokens[:i]] = True
            x = torch.where(seen, torch.where(raw > 0, raw / repetition, raw * repetition), raw)
            x[torch.tensor(s.tokens[n:i], dtype=torch.long).unique()] -= presence
            assert x.max() - x[s.tokens[i]] <= tol, (i, x.max().item(), x[s.tokens[i]].item())
            penalised += (raw.max() - raw[s.tokens[i]] > tol).item()
        single.check()
    assert penalised > 0, "no penalty ever decided"
