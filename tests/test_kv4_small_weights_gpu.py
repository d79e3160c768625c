"""4-bit decode where one row takes nearly all of the softmax and very many others share the rest: the many small
weights add up, so neither the products nor the sums may lose them."""
import math

import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6
VALUE = 6 * 1.625 / 8          # of every element of V but the dominant row's


@pytest.fixture(scope="module")
def gqa():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    from grouped_query_causal_b200 import binding
    binding.load()
    return binding


def _dominated(gqa, hpg, n, k_scale, v_first):
    """Output of sequences of n rows, as many (sequence, KV head) pairs as the GPU takes at a time, so that a pair is
    not split.  Row 0 has K = 7 k_scale (a scale of the format) and V = v_first everywhere, the others K = 0 and V = VALUE;
    all rows but the first 128 lie in one page."""
    Hkv, page = 2, 128
    B = {4: 592, 8: 444, 16: 296}[4 if hpg <= 4 else 8 if hpg <= 8 else 16] // Hkv
    pages = torch.full((2, Hkv, page // 16, ref.RECORD), 0xee, dtype=torch.uint8)      # c = 6
    pages[..., :1024] = 0x88                                                           # c = 0
    pages[..., 2048:] = 12 * 8 + 5                                                     # 1.625 2^-3
    like = pages[0, :, 0].clone()
    for h in range(Hkv):
        ref.put_row(pages, 0, h, 0, torch.full((128,), 7 * k_scale).to(torch.bfloat16), torch.zeros(128).to(torch.bfloat16))
    if v_first == VALUE:
        for at in (slice(1024, 2048), slice(2112, 2176)):
            pages[0, :, 0, at] = like[:, at]
    k, v = ref.unpack(pages[0, :, 0])
    assert (k[:, 0] == 7 * k_scale).all() and (v[:, 0] == v_first).all() and (k[:, 1:] == 0).all() and (v[:, 1:] == VALUE).all()
    tab = torch.ones((B, n // page), dtype=torch.int32)
    tab[:, 0] = 0
    q = torch.ones((B, hpg * Hkv, 128), dtype=torch.bfloat16)
    zeros, lens = torch.zeros(B, dtype=torch.int32), torch.full((B,), n, dtype=torch.int32)
    out = gqa.decode_kv4(q.cuda(), pages.cuda(), tab.cuda(), lens.cuda(), torch.ones(128).cuda(), max_len=n,
                         q_pos=zeros.cuda(), eps=EPS)
    gqa.check_device_status()
    return out.cpu().double()


@pytest.mark.parametrize("hpg", [1, 4, 5, 8, 12, 16])
@pytest.mark.parametrize("k_scale", [1.25 / 8, 1.5 / 8, 1.625 / 8, 1.75 / 8, 1.875 / 8])   # 17.9 to 26.8 base-2 units
def test_weights_far_below_the_largest(gqa, hpg, k_scale):
    """V = 0 in the dominant row: the output is what all the others together weigh."""
    n = 32768
    out = _dominated(gqa, hpg, n, k_scale, 0.0)
    x = 128 * 7 * k_scale / math.sqrt(1 + EPS) / math.sqrt(128)        # the dominant row's logit
    p = math.exp(-x)
    want = VALUE * (n - 1) * p / (1 + (n - 1) * p)
    # logits and sums as in kv_reference.attend: e relative for every weight, 2 e for an output that has one sign; a
    # weight below 2^-16 of the largest is rounded to a multiple of 2^-37 of it
    e = 2.0 ** -19 * x + 2.0 ** -17
    assert (out - want).abs().max() <= 2 * e * want + n * 2.0 ** -38 * VALUE


@pytest.mark.parametrize("hpg", [1, 5, 16])
@pytest.mark.parametrize("k_scale", [1.75 / 8, 1.875 / 8])
def test_sum_of_weights_far_below_the_largest(gqa, hpg, k_scale):
    """The same V in all rows: the output is V, if the sum of the weights holds the small ones as the products do."""
    n = 131072
    out = _dominated(gqa, hpg, n, k_scale, VALUE)
    # A warp has 32768 rows, 512 of them in an accumulator (up to 64 products, each cut off by at most 2^-23 of it) and in
    # a sum of l (up to 32 additions), then 64 such sums, then 12 of lanes and warps, l and O apart: 2^-24 each; 2^-22 for
    # P's two parts, the rescaling by 2^x and the quotient each
    assert (out / VALUE - 1).abs().max() <= 64 * 2.0 ** -23 + (32 + 2 * 64 + 2 * 12) * 2.0 ** -24 + 3 * 2.0 ** -22
