"""Rotary frequencies, and what the operators of a prompt and between the products refuse
before any device work."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import pytest

import speculative_decode_verification_qmm_gb300 as q
from speculative_decode_verification_qmm_gb300 import _lib, build, paged, step

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


# ------------------------------------------------------------------ frequencies
def test_frequencies():
    f, a = q.rope_frequencies(8)
    assert f.dtype == torch.float64 and a == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    g, a = q.rope_frequencies(8, scaling="linear", factor=4)
    assert torch.equal(g, f / 4) and a == 1.0
    g, a = q.rope_frequencies(8, scaling="base", factor=4)
    assert g[0] == 1 and abs(g[3] / f[3] - 0.25) < 1e-14 and a == 1.0
    f, _ = q.rope_frequencies(128, base=1e6)
    g, a = q.rope_frequencies(128, base=1e6, scaling="by parts", factor=8, original_length=4096, slow=2, fast=16)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 16], f[turns >= 16]) and torch.equal(g[turns <= 2], f[turns <= 2] / 8)
    between = (turns > 2) & (turns < 16)
    assert between.any() and ((g < f) & (g > f / 8))[between].all()
    assert a == pytest.approx(0.1 * math.log(8) + 1)


@pytest.mark.parametrize("kw", [dict(dims=0), dict(dims=7), dict(dims=8, base=0.0), dict(dims=8, factor=-1.0), dict(dims=8, scaling="other"),
                                dict(dims=2, scaling="base", factor=2.0), dict(dims=8, scaling="by parts", slow=3.0, fast=3.0)])
def test_frequencies_refused(kw):
    with pytest.raises(ValueError):
        q.rope_frequencies(**kw)


def test_turns_are_the_frequencies():
    """As 64-bit fractions of a turn, whole turns left out, to half a unit."""
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971694, 10 ** 43)
    values = [1.0, 1e-4, 6.5, -0.25, 0.0]
    rope = step.Rope(values, device="cpu")
    for f, t in zip(values, rope.turns.tolist()):
        want = Fraction(f) / two_pi % 1 * (1 << 64)
        assert abs((t % (1 << 64)) - want) <= Fraction(51, 100)
    assert rope.dims == 10


@pytest.mark.parametrize("a,kw", [(([],), {}), (([math.nan],), {}), (([1.0], math.inf), {}), (([1.0],), dict(layout="both"))])
def test_rope_refused(a, kw):
    with pytest.raises(ValueError):
        step.Rope(*a, device="cpu", **kw)


# ------------------------------------------------------------------ the C entries
STRUCTS = ("qmm_rope", "qmm_rotate_args", "qmm_append_args", "qmm_prompt_args", "qmm_norm_args", "qmm_adjust_args", "qmm_attn_args",
           "qmm_sample_args", "qmm_cache_desc")


def test_struct_layouts_match_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "qmm.h"', "int main(void) {"]
    expect = []
    for name in STRUCTS:
        st = getattr(_lib, name)
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        expect.append(ctypes.sizeof(st))
        for f, _ in st._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            expect.append(getattr(st, f).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == expect


def _args(cls, **kw):
    a = cls(struct_size=ctypes.sizeof(cls))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.fixture
def memory():
    return ctypes.addressof(_KEEP)


_KEEP = ctypes.create_string_buffer(4096)


def test_rotate(L, memory):
    m = memory & ~15
    m += 16
    I64 = ctypes.c_int64 * 3

    def call(rope=None, **kw):
        a = _args(_lib.qmm_rotate_args, **(dict(in_dtype=2, out_dtype=0, B=1, T=2, heads=2, turned_heads=1, head_dim=8, x=m, out=m + 512,
                                                x_stride=I64(0, 16, 8), out_stride=I64(0, 16, 8), positions=m) | kw))
        a.rope = _args(_lib.qmm_rope, **(dict(layout=0, dims=8, amplitude=1.0, turns=m) | (rope or {})))
        return L.qmm_rotate(ctypes.byref(a), None)

    assert L.qmm_rotate(None, None) == q.QMM_ERR_INVALID_ARG
    for kw in (dict(struct_size=8), dict(x=None), dict(out=None), dict(positions=None), dict(in_dtype=3), dict(out_dtype=9),
               dict(rope=dict(struct_size=1)), dict(rope=dict(layout=2)), dict(rope=dict(amplitude=math.nan)), dict(rope=dict(turns=None)),
               dict(out=m), dict(out=m, in_dtype=0, out_stride=I64(0, 8, 8))):
        assert call(**kw) == q.QMM_ERR_INVALID_ARG, kw
    for kw in (dict(B=0), dict(T=0), dict(B=65536, T=32768), dict(heads=0), dict(heads=65537), dict(turned_heads=3), dict(turned_heads=-1),
               dict(head_dim=1), dict(head_dim=1025), dict(rope=dict(dims=7)), dict(rope=dict(dims=0)), dict(rope=dict(dims=10))):
        assert call(**kw) == q.QMM_ERR_SHAPE, kw
    for kw in (dict(x=m + 2), dict(out=m + 1), dict(positions=m + 2), dict(rope=dict(turns=m + 4))):
        assert call(**kw) == q.QMM_ERR_ALIGN, kw
    if not torch.cuda.is_available():
        assert call() == q.QMM_ERR_DEVICE


def test_norm(L, memory):
    m = (memory & ~15) + 16

    def call(**kw):
        a = _args(_lib.qmm_norm_args, **(dict(M=2, N=8, res_dtype=0, y_dtype=2, out_dtype=0, eps=1e-6, residual=m, ld_residual=8, y=m + 512, ld_y=8,
                                              residual_out=m, ld_residual_out=8, out=m + 1024, ld_out=8, weight=m, scale=1.0) | kw))
        return L.qmm_residual_norm(ctypes.byref(a), None)

    assert L.qmm_residual_norm(None, None) == q.QMM_ERR_INVALID_ARG
    for kw in (dict(struct_size=8), dict(flags=2), dict(res_dtype=3), dict(y_dtype=3), dict(out_dtype=3), dict(residual=None),
               dict(y=None, out=None), dict(residual_out=None), dict(weight=None), dict(eps=-1.0), dict(eps=math.nan), dict(scale=math.inf),
               # onto one another, and onto inputs that lie otherwise
               dict(out=m), dict(residual_out=m + 1024), dict(ld_residual_out=9), dict(residual_out=m + 512), dict(out=m + 512),
               dict(out=m, y=None, ld_out=9), dict(out=m + 512, y_dtype=1, ld_out=9)):
        assert call(**kw) == q.QMM_ERR_INVALID_ARG, kw
    for kw in (dict(M=0), dict(M=1 << 31), dict(N=0), dict(N=32769)):
        assert call(**kw) == q.QMM_ERR_SHAPE, kw
    for kw in (dict(residual=m + 1), dict(y=m + 2), dict(out=m + 1), dict(weight=m + 2), dict(gate=m + 1), dict(ld_y=7), dict(ld_out=7),
               dict(ld_residual=7), dict(ld_residual_out=0), dict(gate=m, ld_gate=4)):
        assert call(**kw) == q.QMM_ERR_ALIGN, kw
    if not torch.cuda.is_available():
        for kw in (dict(), dict(out=m, y=None), dict(out=m + 512, y_dtype=1), dict(out=m + 512, y_dtype=1, ld_out=9, M=1)):
            assert call(**kw) == q.QMM_ERR_DEVICE


def test_adjust(L, memory):
    m = (memory & ~15) + 16
    I64 = ctypes.c_int64 * 2

    def call(**kw):
        a = _args(_lib.qmm_adjust_args, **(dict(dtype=2, B=2, T=2, V=33, scores=m, stride=I64(66, 33), out=m + 1024, out_stride=I64(66, 33),
                                                counts=m, ld_counts=33, prompt=m, ld_prompt=2) | kw))
        return L.qmm_adjust_scores(ctypes.byref(a), None)

    assert L.qmm_adjust_scores(None, None) == q.QMM_ERR_INVALID_ARG
    for kw in (dict(struct_size=8), dict(dtype=3), dict(scores=None), dict(out=None), dict(out=m, out_stride=I64(33, 66))):
        assert call(**kw) == q.QMM_ERR_INVALID_ARG, kw
    for kw in (dict(B=0), dict(B=65536), dict(T=0), dict(T=65), dict(V=0), dict(V=(1 << 24) + 1)):
        assert call(**kw) == q.QMM_ERR_SHAPE, kw
    for kw in (dict(scores=m + 2), dict(out=m + 2), dict(counts=m + 2), dict(mask=m + 1), dict(bias=m + 2), dict(ld_counts=32), dict(ld_prompt=1),
               dict(bias=m, ld_bias=32)):
        assert call(**kw) == q.QMM_ERR_ALIGN, kw
    if not torch.cuda.is_available():
        assert call() == q.QMM_ERR_DEVICE
    count = lambda **kw: L.qmm_count_tokens(*(dict(counts=m, ld=9, B=2, T=3, V=9, tokens=m, path=m, accept=m, stream=None) | kw).values())  # noqa: E731
    for k in ("counts", "tokens", "path", "accept"):
        assert count(**{k: None}) == q.QMM_ERR_INVALID_ARG
        assert count(**{k: m + 2}) == q.QMM_ERR_ALIGN
    assert count(ld=8) == q.QMM_ERR_ALIGN
    for kw in (dict(B=0), dict(T=65), dict(V=0)):
        assert count(**kw) == q.QMM_ERR_SHAPE


def test_handles(L):
    assert L.qmm_cache_append(None, None, None) == q.QMM_ERR_STATE
    assert L.qmm_prompt_attention(None, None, None) == q.QMM_ERR_STATE
    fake = ctypes.create_string_buffer(256)
    assert L.qmm_prompt_attention(ctypes.addressof(fake), None, None) == q.QMM_ERR_STATE


# ------------------------------------------------------------------ tensors of another GPU
fake = pytest.importorskip("torch._subclasses.fake_tensor")
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU, fake tensors need their device to exist")
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16
APPEND = dict(q=((5, 4, 64), F32), k=((5, 2, 64), F32), v=((5, 2, 64), F32), page_table=((2, 3), I32), lens=((2,), I32), starts=((3,), I32),
              positions=((5,), I32), out=((5, 4, 64), BF16))
PROMPT = dict(q=((5, 4, 64), BF16), page_table=((2, 3), I32), lens=((2,), I32), starts=((3,), I32), out=((5, 4, 64), BF16), lse=((5, 4), F32))
NORM = dict(residual=((3, 8), BF16), y=((3, 8), F32), weight=((8,), F32), bias=((8,), F32), post_weight=((8,), F32), post_bias=((8,), F32),
            gate=((3, 8), F32), out=((3, 8), BF16), residual_out=((3, 8), BF16))
ADJUST = dict(scores=((2, 3, 40), F32), tokens=((2, 3), I32), parents=((2, 3), I32), counts=((2, 40), I32), prompt=((2, 2), I32),
              repetition=((2,), F32), frequency=((2,), F32), presence=((2,), F32), bias=((40,), F32), mask=((2, 3, 2), I32), n_tokens=((2,), I32),
              out=((2, 3, 40), F32))


@pytest.fixture
def cache():
    c = paged.PagedCache.__new__(paged.PagedCache)
    c.handle, c.dtype, c.n_q_heads, c.n_kv_heads, c.head_dim, c._device = None, torch.bfloat16, 4, 2, 64, 0
    return c


def _fakes(where, spec):
    return {n: torch.empty(shape, dtype=dt, device=where.get(n, "cuda:0")) for n, (shape, dt) in spec.items()}


def _refused(call, spec, name):
    with fake.FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
            call(**_fakes({name: "cuda:1"}, spec))
        with pytest.raises(TypeError):
            call(**_fakes({name: "cpu"}, spec))


@no_gpu
@pytest.mark.parametrize("name", APPEND)
def test_append_elsewhere(cache, name):
    _refused(lambda **kw: cache.append(0, **kw), APPEND, name)


@no_gpu
@pytest.mark.parametrize("name", PROMPT)
def test_prompt_elsewhere(cache, name):
    _refused(lambda **kw: cache.attend_prompt(0, **kw), PROMPT, name)


@no_gpu
@pytest.mark.parametrize("name", [n for n in NORM if n != "residual"])
def test_norm_elsewhere(name):
    _refused(q.residual_norm, NORM, name)


@no_gpu
@pytest.mark.parametrize("name", [n for n in ADJUST if n != "scores"])
def test_adjust_elsewhere(name):
    _refused(q.adjust_scores, ADJUST, name)


@no_gpu
def test_rotate_elsewhere():
    rope = step.Rope([1.0], device="cpu")
    rope.device_index = 0
    with fake.FakeTensorMode():
        x, pos = torch.empty(2, 3, 4, 8, device="cuda:0"), torch.empty(2, 3, dtype=I32, device="cuda:0")
        for a in ((x.to("cuda:1"), pos), (x, pos.to("cuda:1"))):
            with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
                rope.rotate(*a)
        for a in ((x.to("cpu"), pos), (x, pos.to("cpu"))):
            with pytest.raises(TypeError):
                rope.rotate(*a)


def test_starts():
    c = paged.PagedCache.__new__(paged.PagedCache)
    c.handle, c.k_pool = None, torch.zeros(1)
    assert c.starts([3, 0, 2]).tolist() == [0, 3, 3, 5] and c.starts([]).tolist() == [0]
    with pytest.raises(ValueError):
        c.starts([1, -1])


# ------------------------------------------------------------------ outputs onto inputs
def _norm_call(L, m, **kw):
    a = _args(_lib.qmm_norm_args, **(dict(M=2, N=8, res_dtype=2, y_dtype=0, out_dtype=0, eps=1e-6, residual=m, ld_residual=8, y=m + 256, ld_y=8,
                                          residual_out=m + 512, ld_residual_out=8, out=m + 768, ld_out=8, weight=m + 1024, scale=1.0,
                                          gate=m + 1280, ld_gate=8) | kw))
    return L.qmm_residual_norm(ctypes.byref(a), None)


@pytest.mark.parametrize("kw", [dict(out="gate"), dict(out="gate", out_dtype=2, ld_out=9), dict(out="gate", out_dtype=2, ld_gate=0),
                                dict(residual_out="gate", ld_residual_out=12), dict(residual_out="gate", ld_gate=0),
                                dict(residual_out="gate", res_dtype=1), dict(out="gate", M=1)])
def test_norm_outputs_onto_a_gate_that_lies_otherwise(L, memory, kw):
    """A row of the output is not the gate's row that its thread reads."""
    m = (memory & ~15) + 16
    kw = {k: m + 1280 if v == "gate" else v for k, v in kw.items()}
    assert _norm_call(L, m, **kw) == q.QMM_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("kw", [dict(out="gate", out_dtype=2), dict(residual_out="gate"), dict(out="gate", out_dtype=2, ld_out=9, M=1),
                                dict(residual_out="gate", ld_gate=0, M=1)])
def test_norm_outputs_onto_a_gate_that_lies_alike(L, memory, kw):
    m = (memory & ~15) + 16
    kw = {k: m + 1280 if v == "gate" else v for k, v in kw.items()}
    assert _norm_call(L, m, **kw) == q.QMM_ERR_DEVICE


@no_gpu
def test_norm_without_y_has_no_gate(L, memory):
    m = (memory & ~15) + 16
    assert _norm_call(L, m, y=None, residual_out=None, out=m + 1280) == q.QMM_ERR_DEVICE
