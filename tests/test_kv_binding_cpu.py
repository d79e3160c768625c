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


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_decode_refuses_what_is_too_short(append, paged, weights):
    """Per-sequence and norm arguments with fewer entries than the kernels read, pages of another head dim."""
    B, H, Hkv, D = 3, 4, 2, 128
    i32 = dict(dtype=torch.int32)
    args = dict(q=_rows(B, H), seqlens=_zeros(B, **i32), qnorm_w=_zeros(D), max_len=16, q_pos=_zeros(B, **i32))
    bad = [dict(seqlens=_zeros(B - 1, **i32)), dict(q_pos=_zeros(B - 1, **i32)), dict(qnorm_w=_zeros(D - 4))]
    if append:
        args.update(k_new=_rows(B, Hkv), v_new=_rows(B, Hkv), knorm_w=_zeros(D))
        bad += [dict(knorm_w=_zeros(D // 2)), dict(v_new=_rows(B - 1, Hkv))]
    if paged:
        pages = _zeros(2, 16, Hkv, D, dtype=torch.bfloat16)
        args.update(k_pages=pages, v_pages=pages, page_table=_zeros(B, 1, **i32))
        narrow = _zeros(2, 16, Hkv, D // 2, dtype=torch.bfloat16)
        bad += [dict(k_pages=narrow, v_pages=narrow), dict(page_table=_zeros(B - 1, 1, **i32))]
    else:
        args.update(k_cache=_rows(48, Hkv), v_cache=_rows(48, Hkv), cache_offsets=_zeros(B + 1, dtype=torch.int64))
        bad += [dict(cache_offsets=_zeros(B, dtype=torch.int64))]
    if weights:
        args.update(weights=_zeros(B, Hkv, 16))
        bad += [dict(weights=_zeros(B - 1, Hkv, 16)), dict(weights=_zeros(B, Hkv, 15))]
    fn = getattr(binding, "decode" + ("_append" if append else "") + ("_paged" if paged else ""))
    for kw in bad:
        with pytest.raises(ValueError) as refusal:
            fn(**{**args, **kw})
        assert "CUDA" not in str(refusal.value), kw        # not because some later tensor is on the CPU
