"""The token-step operators where the range of the numbers or of the bounds is wide: scores far from zero, one token
that outweighs many small ones, elements that outweigh the rest of a vector, bounds far above the lengths."""
import math

import pytest
import torch

from diffusion_transformer_image_mmdit_gb300 import api
from tests import token_oracle as T
from tests.test_gpu_token_ops import (BF16, F64, Seqs, _gpu, device_cache, gen, random_cache, randn, run_attention,
                                      tables, w4_case, within)  # noqa: F401

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


def test_kv_attention_of_a_prompt():
    """Prompts of hundreds of new tokens, alone and behind older ones, units whole and cut."""
    run_attention(gen(61), Seqs(gen(62), [0, 130], [515, 300]), 4, 2, 128)
    run_attention(gen(63), Seqs(gen(64), [0], [400]), 6, 2, 64)


def device_us(f, n=5):
    f()
    best = math.inf
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def test_kv_attention_bounds_far_above_the_lengths():
    """One new token in each of 48 sequences under a bound of 8192 new tokens: the answer of the tight bound, and about its
    time (the merge's grid does not grow with the bound; a factor of 4 and 300 us are left for the launches)."""
    g = gen(65)
    sq = Seqs(g, [int(n) for n in torch.randint(600, 4000, (48,), generator=g)], [1] * 48)
    tokens = random_cache(g, sq.n_blocks, 8, 64)
    k, v, ks, vs = tokens[0] & 0x77, tokens[1] & 0x77, *tokens[2:]
    cache = device_cache(k, v, ks, vs, sq)
    q = randn(g, 48, 32 * 64).to(BF16).cuda()
    took, outs = [], []
    for kw in (dict(), dict(max_new=3, max_len=5000), dict(max_new=8192, max_len=8192)):
        # a table wide enough for the largest bound
        kw["table_ld"] = 128
        wide = api.KVCacheDev(cache.k, cache.v, cache.k_scale, cache.v_scale,
                              torch.nn.functional.pad(cache.table, (0, 128 - cache.table.shape[1])), cache.len, cache.start)
        shape = sq.shape(32, 8, 64, **kw)
        ws, out = api.alloc_workspace(api.kv_workspace_size(shape)), torch.empty_like(q)
        took.append(device_us(lambda: api.mmdit_kv_attention(shape, wide, q, out, ws)))
        outs.append(out.float())
    for o in outs[1:]:
        assert float((o - outs[0]).abs().max()) <= 2.0 ** -6 * float(outs[0].abs().max())
    assert max(took[1:]) <= 4 * took[0] + 300, took


def test_kv_append_bounds_far_above_the_rows():
    """Three rows under a bound of 2^20 new tokens: the cache of the tight bound, and about its time (no sequence has more
    new tokens than there are rows; a factor of 4 and 300 us are left for the launches)."""
    g = gen(66)
    sq = Seqs(g, [300, 5, 64], [1, 1, 1])
    tokens = random_cache(g, sq.n_blocks, 8, 64)
    qkv = randn(g, 3, 48 * 64).to(BF16).cuda()
    cos, sin = tables(400, 64)
    cos, sin = (torch.nn.functional.pad(t, (0, 0, 0, 2 ** 20 - 400)) for t in (cos, sin))
    took, got = [], []
    for max_new in (1, 2 ** 20):
        cache = device_cache(*tokens, sq)
        wide = api.KVCacheDev(cache.k, cache.v, cache.k_scale, cache.v_scale,
                              torch.nn.functional.pad(cache.table, (0, 2 ** 14 - cache.table.shape[1])), cache.len, cache.start)
        shape = sq.shape(32, 8, 64, max_new=max_new, max_len=2 ** 20, table_ld=2 ** 14)
        q = torch.empty(3, 32 * 64, dtype=BF16, device="cuda")
        took.append(device_us(lambda: api.mmdit_kv_append(shape, wide, qkv, cos, sin, q)))
        got.append((q, cache.k, cache.v, cache.k_scale, cache.v_scale))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert took[1] <= 4 * took[0] + 300, took


# ------------------------------------------------------------------ 4-bit products
# A product of an element and a code is exact; a term passes at most 16 sums of an instruction, 8 of a group, K / 1024 + 1
# scaled groups and the parts of 16 warps and 8 blocks, each off by 2^-23 of what is summed (matrix sums cut off).
def exact_tol(x, w, bias, K):
    return 2.0 ** -23 * (16 + 8 + K / 256 + 16) * (x.abs() @ w.abs().t() + bias.abs())


def zero_columns(g, N, K, group, cols):
    w = 0.02 * randn(g, N, K)
    w[:, cols] = 0
    lin = api.quantize_linear_w4(api.LinearDev(w.to(BF16).cuda(), (0.1 * randn(g, N)).cuda()), group)
    w64 = T.w4_weights(lin.w.cpu(), lin.scale.cpu(), group, K)
    assert not w64[:, cols].any()
    return lin, w64


def product(lin, x):
    y = torch.empty(x.shape[0], lin.N, device="cuda")
    api.mmdit_gemv_w4(lin, x.cuda(), y, api.MMDIT_EPI_F32)
    return y.cpu()


@pytest.mark.parametrize("B", [1, 13])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("exp", [10, 20, 40, 120])
def test_gemv_w4_element_that_meets_zero_codes(B, group, exp):
    """Elements far above the rest of their vector whose codes are 0 take nothing from the others' products."""
    g = gen(exp + group)
    K, N, cols = 4096, 200, [7, 1000, 4095]
    lin, w = zero_columns(g, N, K, group, cols)
    x = randn(g, B, K).to(BF16)
    x[:, cols] = torch.tensor([2.0, -2.0, 1.5], dtype=BF16) * 2.0 ** exp
    b = lin.b.cpu().to(F64)
    xx = x.to(F64)
    rest = xx.clone()
    rest[:, cols] = 0
    within(product(lin, x), xx @ w.t() + b, exact_tol(rest, w, b, K), "others")


def test_gemv_w4_elements_of_all_sizes():
    """Vectors whose elements span the range of the type, items of zeros, and the largest and smallest alone."""
    g = gen(70)
    K, N = 2048, 150
    lin, w = w4_case(g, N, K, 64)
    x = (randn(g, 12, K) * torch.exp2(torch.randint(-90, 91, (12, K), generator=g))).to(BF16)
    x[1, 512:] = 0
    x[2, :1024] = 0
    x[3] = (randn(g, K) * 2.0 ** -100).to(BF16)
    x[4], x[5] = 0, 0
    x[4, 600] = 2.0 ** 127
    x[5, 900] = 2.0 ** -100
    x[6] = (randn(g, K) * torch.exp2(torch.randint(0, 40, (K,), generator=g))).to(BF16)
    lin = api.LinearW4Dev(lin.w, lin.scale, 64, K)
    xx = x.to(F64)
    within(product(lin, x), xx @ w.t(), exact_tol(xx, w, torch.zeros(N, dtype=F64), K) * (1 + 1e-9), "sizes")


@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemv_w4_of_unit_vectors_is_the_weights(group):
    """A vector of one element gives a column of W, bit for bit: every code, in every place of a word, in every chunk."""
    g = gen(group)
    K, N = 3 * 128 if group == 128 else 3 * 128 + group, 64
    q = torch.randint(0, 256, (N, api.w4_row_bytes(K)), generator=g).to(torch.uint8)
    s = torch.exp2(randn(g, N, (K + 127) // 128 * (128 // group))).to(BF16)
    lin = api.LinearW4Dev(q.cuda(), s.cuda(), group, K)
    w = T.w4_weights(q, s, group, K)
    for k0 in range(0, K, 16):
        x = torch.zeros(16, K, dtype=BF16)
        x[range(16), range(k0, k0 + 16)] = 1
        assert torch.equal(product(lin, x).to(F64), w[:, k0:k0 + 16].t())


def test_gemv_w4_infinities():
    """An infinity gives what the definition does: an infinity where its code is not 0, a NaN where it is."""
    g = gen(71)
    K, N = 1024, 300
    lin, w = w4_case(g, N, K, 32)
    x = randn(g, 5, K).to(BF16)
    x[0, 3], x[1, 700], x[2, 5], x[2, 900], x[3, 10] = math.inf, -math.inf, math.inf, -math.inf, math.nan
    y, ref = product(lin, x).to(F64), torch.empty(5, N, dtype=F64)
    for i in range(5):
        ref[i] = (x[i].to(F64) * w).sum(1) + lin.b.cpu().to(F64)
    assert bool((w[:, 3] == 0).any()) and bool(torch.isinf(ref[0]).any()) and bool(torch.isnan(ref[0]).any())
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(y), inf) and torch.equal(y[inf], ref[inf])


# ------------------------------------------------------------------ handles
def test_kv_cache_takes_a_slice_of_a_wider_table():
    """The block table of a batch may be rows of a wider one; a bound beyond its columns is refused."""
    g = gen(72)
    sq = Seqs(g, [700, 90, 3], [1, 2, 1], extra_entries=0)
    shape, cache, q, out, _ = run_attention(g, sq, 4, 2, 64, rows_behind=0)
    wide = torch.full((3, 40), -5, dtype=torch.int32, device="cuda")
    wide[:, 4:4 + sq.table_ld] = cache.table
    part = api.KVCacheDev(cache.k, cache.v, cache.k_scale, cache.v_scale, wide[:, 4:4 + sq.table_ld], cache.len, cache.start)
    got = attend(sq.shape(4, 2, 64, table_ld=40), part, q)
    assert torch.equal(got, out.cpu())
    # one sequence of it, under either row length
    one = api.KVCacheDev(cache.k, cache.v, cache.k_scale, cache.v_scale, wide[:1, 4:4 + sq.table_ld], cache.len[:1].clone(),
                         cache.start[:2].clone())
    for ld in (40, sq.table_ld):
        got = attend(sq.shape(4, 2, 64, B=1, n_new=1, max_new=1, table_ld=ld), one, q[:1]).float()
        # another batch is cut in other places, and rounds differently
        assert float((got - out[:1].cpu().float()).abs().max()) <= 2.0 ** -6 * float(got.abs().max())
    with pytest.raises(ValueError):
        attend(sq.shape(4, 2, 64, table_ld=40, max_len=sq.table_ld * 64 + 1), part, q)
    with pytest.raises(ValueError):
        attend(shape, part, q)  # the table's own stride
    with pytest.raises(ValueError):
        api.KVCacheDev(cache.k, cache.v, cache.k_scale, cache.v_scale, wide.t()[:3], cache.len, cache.start)
