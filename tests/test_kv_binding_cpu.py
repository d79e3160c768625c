"""Tensors that the Python binding refuses on the host, before the library is called (no GPU: tensors that claim to
be on one)."""
import pytest
import torch

from grouped_query_causal_b200 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


class _Claims(torch.Tensor):
    is_cuda = True


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Claims)


def _rows(n, Hkv, D=128):
    return _zeros(n, Hkv, D, dtype=torch.bfloat16)


def test_rows_that_overlap_are_refused():
    n, Hkv = 5, 2
    for bad in (_rows(1, Hkv).expand(n, Hkv, 128), _rows(n, 1).expand(n, Hkv, 128),
                torch.as_strided(_rows(n, Hkv), (n, Hkv, 128), (128, 128, 1)).as_subclass(_Claims)):
        with pytest.raises(ValueError):
            binding._check_rows(bad, "k_hat", n, Hkv)
        pages, tab = _zeros(1, Hkv, 1, binding.KV4_RECORD_BYTES, dtype=torch.uint8), _zeros(1, 1, dtype=torch.int32)
        cu, pre = _zeros(2, dtype=torch.int64), _zeros(1, dtype=torch.int32)
        good = _rows(n, Hkv)
        for k, v in ((bad, good), (good, bad)):
            with pytest.raises(ValueError):
                binding.kv4_write(k, v, cu, pre, pages, tab)
            with pytest.raises(ValueError):
                binding.kv4_read(pages, tab, cu, pre, n, k_out=k, v_out=v)
    assert binding._check_rows(_rows(n, Hkv), "k_hat", n, Hkv) == Hkv * 128
    assert binding._check_rows(_rows(1, Hkv).expand(1, Hkv, 128), "k_hat", 1, Hkv) == Hkv * 128
    wide = _zeros(n, 3 * 128, dtype=torch.bfloat16)[:, :Hkv * 128].unflatten(1, (Hkv, 128))
    assert binding._check_rows(wide, "k_hat", n, Hkv) == 3 * 128
    assert binding._check_rows(_rows(0, Hkv), "k_hat", 0, Hkv) == Hkv * 128
