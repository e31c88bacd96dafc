"""What the paged cache's Python calls refuse before any device work: tensors of
another GPU than the pools', by tensors that have a device and no memory."""
import pytest

from speculative_decode_verification_qmm_gb300 import paged

torch = pytest.importorskip("torch")
fake = pytest.importorskip("torch._subclasses.fake_tensor")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU, fake tensors need their device to exist")


@pytest.fixture
def cache():
    c = paged.PagedCache.__new__(paged.PagedCache)
    c.handle, c.dtype, c.n_q_heads, c.n_kv_heads, c.head_dim, c._device = None, torch.bfloat16, 4, 2, 64, 0
    return c


def _args(where, spec):
    """Fake tensors of `spec` (name: shape, dtype), those named in `where` on a device of their own."""
    return {n: torch.empty(shape, dtype=dt, device=where.get(n, "cuda:0")) for n, (shape, dt) in spec.items()}


I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16
ATTEND = dict(q=((2, 3, 4, 64), BF16), k=((2, 3, 2, 64), BF16), v=((2, 3, 2, 64), BF16), page_table=((2, 5), I32),
              lens=((2,), I32), mask=((2, 3), torch.int64), n_tokens=((2,), I32), out=((2, 3, 4, 64), BF16),
              lse=((2, 3, 4), F32))
COMMIT = dict(page_table=((2, 5), I32), lens=((2,), I32), path=((2, 3), I32), accept=((2, 2), I32), lens_out=((2,), I32))
COPY = dict(src=((3,), I32), dst=((3,), I32), rows=((3,), I32))
SAMPLE = dict(target=((2, 3, 9), F32), draft=((2, 3, 9), F32), tokens=((2, 3), I32), u=((2, 3), F32), noise=((2, 9), F32),
              parents=((2, 3), I32), temperature=((2,), F32), n_tokens=((2,), I32))


@pytest.mark.parametrize("name", ATTEND)
def test_attend(cache, name):
    with fake.FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
            cache.attend(0, **_args({name: "cuda:1"}, ATTEND))
        with pytest.raises(TypeError):
            cache.attend(0, **_args({name: "cpu"}, ATTEND))


@pytest.mark.parametrize("name", COMMIT)
def test_commit(cache, name):
    with fake.FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
            cache.commit(**_args({name: "cuda:1"}, COMMIT))
        with pytest.raises(TypeError):
            cache.commit(**_args({name: "cpu"}, COMMIT))


@pytest.mark.parametrize("name", COPY)
def test_copy_pages(cache, name):
    with fake.FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
            cache.copy_pages(**_args({name: "cuda:1"}, COPY))
        with pytest.raises(TypeError):
            cache.copy_pages(**_args({name: "cpu"}, COPY))


@pytest.mark.parametrize("name", [n for n in SAMPLE if n != "target"])
def test_verify_sample(name):
    with fake.FakeTensorMode():
        with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
            paged.verify_sample(**_args({name: "cuda:1"}, SAMPLE))
        with pytest.raises(TypeError):
            paged.verify_sample(**_args({name: "cpu"}, SAMPLE))


def test_pools():
    with fake.FakeTensorMode():
        pools = _args({"v_pool": "cuda:1"}, dict(k_pool=((1, 2, 1, 16, 64), BF16), v_pool=((1, 2, 1, 16, 64), BF16)))
        with pytest.raises(ValueError, match="cuda:0, not cuda:1"):
            paged.PagedCache(1, 2, 16, 1, 1, 64, **pools)
        pools = _args({"k_pool": "cpu", "v_pool": "cpu"}, dict(k_pool=((1, 2, 1, 16, 64), BF16), v_pool=((1, 2, 1, 16, 64), BF16)))
        with pytest.raises(TypeError):
            paged.PagedCache(1, 2, 16, 1, 1, 64, **pools)
