"""The paged cache's host side, without a GPU: struct layouts, argument validation
that comes before any device work, and the page bookkeeping."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import speculative_decode_verification_qmm_gb300 as q
from speculative_decode_verification_qmm_gb300 import _lib, build, paged

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.load()


def test_struct_layouts_match_header(tmp_path):
    structs = (_lib.qmm_cache_desc, _lib.qmm_attn_args, _lib.qmm_sample_args)
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "qmm.h"', "int main(void) {"]
    want = []
    for st in structs:
        lines.append(f'printf("%zu\\n", sizeof({st.__name__}));')
        want.append(ctypes.sizeof(st))
        for f, _ in st._fields_:
            lines.append(f'printf("%zu\\n", offsetof({st.__name__}, {f}));')
            want.append(getattr(st, f).offset)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def test_host_validation_without_device(L):
    assert q.qmm_strerror(9) == "QMM_ERR_INDEX"
    h = ctypes.c_void_p(7)
    assert L.qmm_cache_create(None, None, None) == q.QMM_ERR_INVALID_ARG
    assert L.qmm_cache_create(ctypes.byref(h), None, None) == q.QMM_ERR_INVALID_ARG and h.value is None
    d = _lib.qmm_cache_desc(8, 0, 1, 16, 2, 1, 64, 1, 4, 4096, 4096)
    assert L.qmm_cache_create(ctypes.byref(h), ctypes.byref(d), None) == q.QMM_ERR_INVALID_ARG
    d.struct_size = ctypes.sizeof(d)
    for field, value, code in (("dtype", 2, q.QMM_ERR_INVALID_ARG), ("k_pool", None, q.QMM_ERR_INVALID_ARG),
                               ("page_size", 17, q.QMM_ERR_SHAPE), ("head_dim", 32, q.QMM_ERR_SHAPE),
                               ("n_pages", 1 << 31, q.QMM_ERR_SHAPE), ("v_pool", 4100, q.QMM_ERR_ALIGN)):
        bad = _lib.qmm_cache_desc.from_buffer_copy(d)
        setattr(bad, field, value)
        assert L.qmm_cache_create(ctypes.byref(h), ctypes.byref(bad), None) == code, field
    fake = ctypes.create_string_buffer(512)
    a = _lib.qmm_attn_args()
    assert L.qmm_tree_attention(None, ctypes.byref(a), None) == q.QMM_ERR_STATE
    assert L.qmm_tree_attention(ctypes.addressof(fake), ctypes.byref(a), None) == q.QMM_ERR_STATE
    assert L.qmm_cache_commit(None, 1, 1, None, 1, 1, None, None, 1, None, None, None) == q.QMM_ERR_STATE
    assert L.qmm_cache_copy(None, 0, None, None, None, None) == q.QMM_ERR_STATE
    assert L.qmm_cache_sync_status(None, None) == q.QMM_ERR_STATE
    assert L.qmm_cache_destroy(None) == q.QMM_OK
    assert L.qmm_cache_destroy(ctypes.addressof(fake)) == q.QMM_ERR_STATE
    s = _lib.qmm_sample_args()
    assert L.qmm_verify_sample(ctypes.byref(s), None) == q.QMM_ERR_INVALID_ARG
    n = ctypes.c_int64()
    assert L.qmm_verify_sample_workspace(2, 8, 1000, ctypes.byref(n)) == q.QMM_OK and n.value > 0


class Book(paged.PagedCache):
    """The bookkeeping alone: copies are recorded, not made."""

    def __init__(self, n_pages, page_size):
        self.n_pages, self.page_size, self.handle = n_pages, page_size, None
        self.k_pool = torch.zeros(1)
        self._users, self._free = [0] * n_pages, list(range(n_pages - 1, -1, -1))
        self.copied = []

    def _copy(self, copies, stream=None):
        self.copied += copies

    def consistent(self, seqs):
        users = [0] * self.n_pages
        for s in seqs:
            assert len(s.pages) == len(set(s.pages))
            for p in s.pages:
                users[p] += 1
        assert users == self._users
        assert sorted(self._free) == [p for p in range(self.n_pages) if users[p] == 0]


def test_reserve_fork_free():
    c = Book(10, 16)
    a = c.new_sequence()
    c.reserve([a], 40)
    assert len(a.pages) == 3 and c.free_pages == 7
    c.advance([a], [40])
    b = c.fork(a)
    assert b.pages == a.pages and b.length == 40 and c.free_pages == 7
    c.reserve([a, b], 1)  # the last page is shared: the first of the two copies it
    assert a.pages[:2] == b.pages[:2] and a.pages[2] != b.pages[2]
    assert len(c.copied) == 1 and c.copied[0] == (b.pages[2], a.pages[2], 8)
    c.consistent([a, b])
    c.advance([a, b], [8, 3])
    d = c.fork(a)  # 48 rows: three full pages, nothing to copy
    c.reserve([d], 16)
    assert len(c.copied) == 1 and d.pages[:3] == a.pages and len(d.pages) == 4
    c.consistent([a, b, d])
    c.free(a)
    c.consistent([b, d])
    c.free(b)
    c.free(d)
    c.consistent([])
    assert c.free_pages == 10


def test_reserved_pages_are_not_forked():
    """Pages past the cached rows belong to the sequence that reserved them."""
    c = Book(6, 16)
    a = c.new_sequence()
    c.reserve([a], 40)
    c.advance([a], [16])
    b = c.fork(a)
    assert b.pages == a.pages[:1]
    c.reserve([b], 1)
    assert b.pages[0] == a.pages[0] and b.pages[1] not in a.pages and c.copied == []
    c.consistent([a, b])


def test_too_few_pages_takes_none():
    c = Book(3, 16)
    a, b = c.new_sequence(), c.new_sequence()
    with pytest.raises(MemoryError):
        c.reserve([a, b], 32)
    assert a.pages == [] and b.pages == [] and c.free_pages == 3
    c.reserve([a], 33)
    with pytest.raises(ValueError):
        c.advance([a], [49])
    c.advance([a], [40])
    f = c.fork(a)
    with pytest.raises(MemoryError):
        c.reserve([f], 1)
    c.consistent([a, f])


def test_random_bookkeeping():
    r = np.random.default_rng(0)
    c = Book(60, 16)
    seqs = []
    for _ in range(2000):
        what = r.integers(0, 4)
        if what == 0 and len(seqs) < 12:
            seqs.append(c.new_sequence())
        elif what == 1 and seqs:
            some = [s for s in seqs if r.random() < 0.5]
            rows = int(r.integers(1, 40))
            before = [(list(s.pages), s.length) for s in seqs]
            try:
                c.reserve(some, rows)
            except MemoryError:
                assert before == [(s.pages, s.length) for s in seqs]
            else:
                for s in some:
                    assert len(s.pages) * 16 >= s.length + rows
                    assert all(c._users[p] == 1 for p in s.pages[s.length // 16:])
                c.advance(some, [int(r.integers(0, rows + 1)) for _ in some])
        elif what == 2 and seqs and len(seqs) < 12:
            seqs.append(c.fork(seqs[r.integers(len(seqs))]))
        elif seqs:
            c.free(seqs.pop(r.integers(len(seqs))))
        c.consistent(seqs)


def test_tree_mask():
    m = q.tree_mask(torch.tensor([[-1, 0, 0, 1, 3], [-1, -1, 0, 1, 2]]))
    assert m.tolist() == [[1, 3, 5, 11, 27], [1, 2, 5, 10, 21]]
    chain = q.tree_mask(torch.arange(-1, 63)[None])
    assert chain[0, 63] == -1 and chain[0, 62] == (1 << 63) - 1
    with pytest.raises(ValueError):
        q.tree_mask(torch.tensor([[0]]))


def test_sample_workspace_holds_for_any_gpu(L):
    """Every row has room for all of its parts, 4,096 entries each and 32 at most,
    whatever share of them a GPU's number of SMs makes a call use."""
    for V, parts in ((1, 1), (4097, 2), (151936, 32)):
        one = q.qmm_verify_sample_workspace(1, 8, V)
        assert one == 8 * 2 * parts * 8
        assert q.qmm_verify_sample_workspace(40, 8, V) == 40 * one
