"""The token-step operators where the range of the numbers or of the bounds is wide: scores far from zero, one token
that outweighs many small ones, elements that outweigh the rest of a vector, bounds far above the lengths."""
import pytest
import torch

from diffusion_transformer_image_mmdit_gb300 import api
from tests import token_oracle as T
from tests.test_gpu_token_ops import (BF16, F64, Seqs, _gpu, device_cache, gen, random_cache, randn,
                                      within)  # noqa: F401

pytestmark = pytest.mark.gpu


def attend(shape, cache, q):
    out = torch.empty(q.shape[0], shape.H * shape.d_head, dtype=BF16, device="cuda")
    api.mmdit_kv_attention(shape, cache, q.cuda(), out, api.alloc_workspace(api.kv_workspace_size(shape)))
    return out.cpu()


def value_codes(v):
    """[..., d, 64] codes of values [..., 64, d]."""
    return T.e4m3(v).transpose(-1, -2).contiguous()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("tokens", [300, 8192])
@pytest.mark.parametrize("j", [12, 17, 19, 21, 24, 52, 80])
@pytest.mark.parametrize("q0", [1.3828125, -1.7265625])
def test_kv_attention_scores_far_above_one(tokens, j, q0):
    """Scores of some 2^8 2^j: the token with the largest alone is left, whatever the rounding of its score, or, where
    two have it, their mean.  The next largest lies 2^-10 of it below (scores carry 2^-19 of the products' sum)."""
    g = gen(j)
    sq = Seqs(g, [tokens - 1], [1])
    k, v, _, _ = random_cache(g, sq.n_blocks, 1, 64)
    k, v = k & 0xB7, v & 0xB7  # finite, below 1
    top = [sq.table[0][at // 64] for at in (70, 260)]
    slot = [70 % 64, 260 % 64]
    ks, vs = torch.full((sq.n_blocks, 1), 2.0 ** j), torch.ones(sq.n_blocks, 1)
    best = torch.randint(0x40, 0x58, (64,), generator=g).to(torch.uint8) | (0x80 if q0 < 0 else 0)
    k[top[0], 0, slot[0]] = best
    two = tokens == 8192  # the same score once more, in another block of another scale
    if two:
        ks[top[1]] = 2.0 ** (j - 1)
        k[top[1], 0] = 0
        k[top[1], 0, slot[1]] = best + 8  # twice the value
    cache = T.Cache(k, v, ks, vs)
    kk, vv = cache.rows(sq.table[0], 0, tokens)
    s = (kk * q0).sum(1)
    first = s.sort(descending=True).values
    assert float(first[2 if two else 1]) < float(first[0]) * (1 - 2.0 ** -10) and s[70] == first[0]
    shape = sq.shape(2, 1, 64)
    out = attend(shape, device_cache(k, v, ks, vs, sq), torch.full((1, 128), q0, dtype=BF16))
    want = (vv[70] + vv[260]) / 2 if two else vv[70]
    for h in range(2):
        within(out.view(2, 64)[h], want, (2.0 ** -8 + 2.0 ** -18) * want.abs(), "one token")


@pytest.mark.parametrize("tokens", [300, 8192, 65537])
@pytest.mark.parametrize("nats", [12, 16, 18, 22])
@pytest.mark.parametrize("d", [64, 128])
def test_kv_attention_one_token_above_many(tokens, nats, d):
    """One token (its value 0) stands `nats` above all others, which share the rest: what they give is the output.  P is
    rounded to f16, half a step 2^-11, or 2^-39 of the largest p where that is more; scores carry 2^-19 of their
    magnitude and P's sums 2^-18; the output is rounded to bf16, 2^-8."""
    g = gen(nats)
    sq = Seqs(g, [tokens - 1], [1])
    code = int(T.e4m3(torch.tensor([-2.0 * nats]))[0])
    assert float(T.e4m3_value(torch.tensor([code], dtype=torch.uint8))) == -2 * nats
    k = torch.full((sq.n_blocks, 1, 64, d), code, dtype=torch.uint8)
    v = value_codes(1 + torch.rand(sq.n_blocks, 1, 64, d, generator=g))
    blk = sq.table[0][1]
    k[blk, 0, 5], v[blk, 0, :, 5] = 0, 0
    ks, vs = torch.full((sq.n_blocks, 1), 0.5), torch.ones(sq.n_blocks, 1)
    out = attend(sq.shape(4, 1, d, scale=1.0 / d), device_cache(k, v, ks, vs, sq), torch.ones(1, 4 * d, dtype=BF16))
    kk, vv = T.Cache(k, v, ks, vs).rows(sq.table[0], 0, tokens)
    p = torch.softmax(kk.mean(1), 0)
    o = p @ vv
    tol = 2.0 ** -8 * o + (2.0 ** -11 + 2.0 ** -18 + nats * 2.0 ** -19) * 1.01 * o + tokens * 2.0 ** -39 * 2 * p.max()
    for h in range(4):
        within(out.view(4, d)[h], o, tol, "the many")


@pytest.mark.parametrize("d", [64, 128])
def test_kv_attention_query_channel_that_meets_zero_keys(d):
    """A channel of the queries 2^20 above the others, whose keys are 0, takes nothing from the others' products."""
    g = gen(d)
    sq = Seqs(g, [255], [1])
    k, v = T.e4m3(randn(g, sq.n_blocks, 1, 64, d)), T.e4m3(randn(g, sq.n_blocks, 1, d, 64))
    k[..., 9] = 0
    ks = vs = torch.ones(sq.n_blocks, 1)
    q = randn(g, 1, 2 * d).to(BF16)
    q.view(2, d)[:, 9] = 2.0 ** 20
    out = attend(sq.shape(2, 1, d), device_cache(k, v, ks, vs, sq), q)
    kk, vv = T.Cache(k, v, ks, vs).rows(sq.table[0], 0, 256)
    qq = q.view(2, d).to(F64)
    p = torch.softmax(qq @ kk.t() * d ** -0.5, 1)
    o, mag = p @ vv, (qq.abs() @ kk.abs().t() * d ** -0.5).amax(1, keepdim=True)
    tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -18 + mag * 2.0 ** -19) * 1.01 * (p @ vv.abs()) + 256 * 2.0 ** -39 * vv.abs().amax()
    within(out.view(2, d), o, tol, "outlier channel")
