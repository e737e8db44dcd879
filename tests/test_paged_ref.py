"""Pins of the 64-bit forms that the paged serving operators are tested with: against PyTorch's float64 attention and the
oracle's prologue on caches that pages only rearrange, hand-worked cases, and defining properties. No GPU."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_ref as R


def _flat(b, s):
    """Keys and values of sequence s by its block table, from the pools as stored."""
    out = []
    for pool, sc in ((b.k, b.ks), (b.v, b.vs)):
        pos = torch.arange(b.kv[s])
        x = pool.float().double()[b.table[s, pos // b.page].long(), pos % b.page]
        out.append(x if sc is None else x * sc.double()[:, None])
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("window", [0, 1, 7, 40])
@pytest.mark.parametrize("hq,hkv,page", [(4, 4, 16), (6, 2, 32), (3, 1, 16)])
def test_attention_is_torchs(hq, hkv, page, window, e4m3):
    b = R.Paged(hq + page, [1, 0, 9, 33], [50, 3, 9, 70], hq, hkv, page, e4m3, pad=2, device="cpu")
    got = R.attention(b, window)
    for s in range(b.B):
        n, kv, r0 = b.new[s], b.kv[s], int(b.q_start[s])
        k, v = (x.repeat_interleave(hq // hkv, 1).permute(1, 0, 2)[None] for x in _flat(b, s))
        q = b.q[r0:r0 + n].double().permute(1, 0, 2)[None]
        pos, j = torch.arange(kv - n, kv)[:, None], torch.arange(kv)[None]
        sees = (j <= pos) & ((j > pos - window) if window else True)
        if n == 0:
            continue
        want = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=sees)[0].permute(1, 0, 2)
        assert (got[r0:r0 + n] - want).abs().max() < 1e-12
    assert (got[b.rows:] == 0).all()


def test_attention_of_one_visible_key_is_its_value():
    b = R.Paged(1, [3], [20], 4, 2, 16, device="cpu")
    k, v = _flat(b, 0)
    got = R.attention(b, window=1)
    for i in range(3):
        for h in range(4):
            assert torch.equal(got[i, h], v[17 + i, h // 2])


def test_attention_counts_invalid_pages_as_zeros():
    b = R.Paged(2, [1], [48], 2, 1, 16, device="cpu")
    whole = _flat(b, 0)
    b.table[0, 1] = b.n_pages
    k, v = b.values(0)
    for x, w in ((k, whole[0]), (v, whole[1])):
        assert (x[16:32] == 0).all()
        assert torch.equal(x[:16], w[:16]) and torch.equal(x[32:], w[32:])


@pytest.mark.parametrize("rope", [False, True])
def test_append_is_the_oracles_prologue(rope):
    b = R.Paged(3, [5, 1, 4], [9, 30, 4], 6, 2, 16, device="cpu")
    g = torch.Generator().manual_seed(1)
    qw, kw = ((torch.rand(R.DH, generator=g) + 0.5).to(torch.bfloat16) for _ in range(2))
    a = torch.rand((40, 64), generator=g) * 6
    cs = torch.cat([a.cos(), a.sin()], 1).float()
    bits = lambda x: x.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    pos = np.array([p for n, kv in zip(b.new, b.kv) for p in range(kv - n, kv)], np.int32)
    q, k, v = oracle.qk_norm_rope_kv(bits(b.qkv), 6, 2, bits(qw), bits(kw), cs.numpy() if rope else None,
                                     pos if rope else None, rope, 1e-6)
    (mq, _), (mk, _), mv = R.append(b, qw, kw, cs, 1e-6, rope)
    for mine, want in ((mq, q), (mk, k), (mv, v)):
        assert np.abs(mine.numpy() - np.asarray(want, np.float64).reshape(mine.shape)).max() < 1e-12


def test_append_by_hand():
    b = R.Paged(4, [1], [3], 1, 1, 16, device="cpu")
    b.qkv[:] = 0
    b.qkv[0, 0, 0], b.qkv[0, 1, 64] = 2.0, 4.0
    cs = torch.zeros(3, R.DH)
    cs[2, 64:] = 1.0  # a quarter turn at position 2
    one = torch.ones(R.DH, dtype=torch.bfloat16)
    (q, _), (k, _), _ = R.append(b, None, None, cs, 0.0, True)
    assert q[0, 0, 64] == 2.0 and q[0, 0].abs().sum() == 2.0       # (x, 0) -> (0, x)
    assert k[0, 0, 0] == -4.0 and k[0, 0].abs().sum() == 4.0       # (0, x) -> (-x, 0)
    (q, _), _, _ = R.append(b, one, one, cs, 0.0, False)
    assert abs(float(q[0, 0, 0]) - math.sqrt(R.DH)) < 1e-12        # one element of 128: its RMS is x / sqrt(128)


LOG = [0.0, math.log(2), math.log(4), -math.inf, math.log(2)]  # weights 1/4, 1/2, 1, none, 1/2 of the largest


@pytest.mark.parametrize("t,k,p,m,u,token,share", [
    (1.0, 0, 1.0, 0.0, 0.0, 0, 1 / 9), (1.0, 0, 1.0, 0.0, 0.12, 1, 2 / 9), (1.0, 0, 1.0, 0.0, 0.5, 2, 4 / 9),
    (1.0, 0, 1.0, 0.0, 0.99, 4, 2 / 9), (0.0, 0, 1.0, 0.0, 0.99, 2, 1.0),
    (1.0, 2, 1.0, 0.0, 0.0, 1, 1 / 3),      # the lower index of the two equals
    (1.0, 2, 1.0, 0.0, 0.9, 2, 2 / 3),
    (1.0, 3, 0.5, 0.0, 0.9, 2, 1.0),        # half of the first three's mass is the largest alone
    (1.0, 3, 0.51, 0.0, 0.0, 1, 1 / 3), (1.0, 0, 0.0, 0.0, 0.5, 2, 1.0),
    (1.0, 0, 1.0, 0.5, 0.0, 1, 1 / 4),      # 1/4 is below min-p
    (1.0, 0, 1.0, 2.0, 0.7, 2, 1.0),        # the largest always stays
    (0.5, 0, 1.0, 0.0, 0.0, 0, 1 / 25), (math.inf, 0, 1.0, 0.0, 0.6, 2, 1 / 4)])
def test_sample_by_hand(t, k, p, m, u, token, share):
    got, lp = R.sample(torch.tensor(LOG, dtype=torch.float64), t, k, p, m, u)
    assert got == token and abs(lp - math.log(share)) < 1e-12


def test_sample_draws_in_proportion():
    # over a grid of u, each token as often as its share of what the filters keep
    x = torch.randn(40, generator=torch.Generator().manual_seed(5), dtype=torch.float64) * 2
    x[7] = -math.inf
    n = 4000
    for t, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 9, 1.0, 0.0), (1.3, 0, 0.8, 0.0), (1.0, 20, 0.9, 0.05)):
        counts = np.zeros(40)
        share = {}
        for i in range(n):
            tok, lp = R.sample(x, t, k, p, m, (i + 0.5) / n)
            counts[tok] += 1
            share[tok] = math.exp(lp)
        assert abs(sum(share.values()) - 1) < 1e-9
        assert all(abs(counts[i] / n - share.get(i, 0.0)) <= 1.5 / n for i in range(40))
        if k:
            assert len(share) <= k
        kept = torch.tensor(sorted(share))
        w = torch.exp((x - x.max()) / t)
        assert float(w[kept].min()) >= m
        assert float(x[kept].min()) >= float(x[[i for i in range(40) if i not in share]].max())


def test_sample_nothing():
    for row in ([-math.inf] * 3, [math.nan] * 3):
        assert R.sample(torch.tensor(row, dtype=torch.float64), 1.0, 0, 1.0, 0.0, 0.5) == (-1, -math.inf)
