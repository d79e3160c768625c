"""4-bit decode with append and accumulated weights where a KV head has 5 to 8, 9 to 16 and more query heads (several
passes over the same records, one of which stores the new row), with scaled RoPE, against the forms of kv_reference."""
import math

import pytest
import torch

from tests import kv_reference as ref

pytestmark = pytest.mark.gpu
EPS, THETA = 1e-6, 1.0e6
YARN = dict(scaling="yarn", factor=16.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0)


@pytest.fixture(scope="module")
def gqa():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA device is required for the gpu tests")
    from grouped_query_causal_b200 import binding
    binding.load()
    return binding


def _hat(x, w, pos, pairing, scaled):
    """ref.hat, or with YaRN's frequencies (its logit factor is not in here)."""
    if not scaled:
        return ref.hat(x, w, pos, EPS, theta=THETA, pairing=pairing)
    x = x.double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
    f = THETA ** (-2.0 * torch.arange(64, dtype=torch.float64) / 128)
    turns = YARN["original_max_position"] * f / (2 * math.pi)
    keep = ((turns - YARN["beta_slow"]) / (YARN["beta_fast"] - YARN["beta_slow"])).clamp(0, 1)
    a = float(pos) * f * ((1 - keep) / YARN["factor"] + keep)
    c, s = torch.cos(a), torch.sin(a)
    lo, hi = (slice(0, 64), slice(64, 128)) if pairing == "half" else (slice(0, 128, 2), slice(1, 128, 2))
    out = torch.empty_like(y)
    out[..., lo], out[..., hi] = y[..., lo] * c - y[..., hi] * s, y[..., lo] * s + y[..., hi] * c
    return out


@pytest.mark.parametrize("H,Hkv,page,pairing", [(16, 2, 16, "adjacent"), (10, 2, 64, "half"), (33, 1, 48, "adjacent"),
                                                (40, 2, 32, "half"), (4, 1, 16, "half")])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("append", [False, True])
def test_forms(gqa, H, Hkv, page, pairing, scaled, append):
    g = torch.Generator()
    g.manual_seed(H + page)
    lens = [0 if append else 1, 1, 15, 16, 31, 32, 63, 64, 500, 3001]
    B, add = len(lens), 1 if append else 0
    tab, num = ref.page_table([n + add for n in lens], page, g, spare=1)
    pages = ref.random_pages(num, page, Hkv, g)
    q, kn, vn = (torch.randn((B, h, 128), generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv))
    wq, wk = torch.rand(128, generator=g) + 0.5, torch.rand(128, generator=g) + 0.5
    at = [n + 5000 * (b % 3) for b, n in enumerate(lens)]
    room = max(lens) + add
    weights = torch.rand((B, Hkv, room + 2), generator=g)
    w, pos = weights.cuda(), torch.full(weights.shape, -5, dtype=torch.int32, device="cuda")
    got, sl = pages.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    kw = dict(max_len=room, q_pos=torch.tensor(at, dtype=torch.int32).cuda(), eps=EPS,
              rope=gqa.RopeConfig.make(theta=THETA, pairing=pairing, **(YARN if scaled else {})), weights=w)
    if append:
        out = gqa.decode_append_kv4(q.cuda(), kn.cuda(), vn.cuda(), got, tab.cuda(), sl, wq.cuda(), wk.cuda(), row_pos=pos, **kw)
    else:
        out = gqa.decode_kv4(q.cuda(), got, tab.cuda(), sl, wq.cuda(), **kw)
    gqa.check_device_status()
    factor = (0.1 * math.log(YARN["factor"]) + 1) ** 2 if scaled else 1.0
    for b, n in enumerate(lens):
        if append:
            kh = _hat(kn[b], wk, at[b], pairing, scaled).float().to(torch.bfloat16)
            for h in range(Hkv):
                ref.put_row(pages, int(tab[b, n // page]), h, n % page, kh[h], vn[b, h])
        m = n + add
        k, v = ref.rows4(pages, tab, b, m)
        want, got_w, tol, wtol = ref.attend(factor * _hat(q[b], wq, at[b], pairing, scaled), k, v)
        assert (out[b].cpu().double() - want).abs().max() <= tol, b
        total = weights[b].double()
        if append:
            total[:, n] = 0
            assert (pos[b, :, n] == at[b]).all()
        assert (pos[b] != -5).sum() == Hkv * add
        total[:, :m] += got_w
        err = (w[b].cpu().double() - total).abs()
        # 2^-24 of the sum for each of the H / Hkv additions and the last one
        assert (err[:, :m] <= wtol + 2.0 ** -24 * (H // Hkv + 1) * total[:, :m]).all(), b
        assert (err[:, m:] == 0).all()
    assert torch.equal(got.cpu(), pages)          # exactly the new rows were written
