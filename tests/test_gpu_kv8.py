"""The 8-bit KV cache on the GPU: append, read back and attention against plain implementations in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import decode_persistent_megakernel_gb300 as T  # noqa: E402
import kv8_ref as R  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu
E4M3, INT8 = T.TINFER_KV8_E4M3, T.TINFER_KV8_INT8
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    T.build()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(shape, seed, scale=1.0):
    return scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def garbage(cache, seed=0):
    """Fills a cache with what a reader must not see: random codes (NaN codes of e4m3 among them) and scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for c in (cache.k_codes, cache.v_codes):
        c.copy_(torch.randint(0, 256, c.shape, generator=g, device="cuda", dtype=torch.uint8))
    for s in (cache.k_scales, cache.v_scales):
        s.copy_(torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.5, math.nan, 1e30))


def filled(heads, d, lens, max_ctx, fmt, block, seed, spread=1.0):
    """A cache whose sequence s holds lens[s] tokens with scales of its own per block, garbage behind them."""
    cache = T.Kv8Cache(heads, d, max_ctx, n_seqs=len(lens), fmt=fmt, block=block)
    garbage(cache, seed)
    g = torch.Generator().manual_seed(seed)
    for codes, scales in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        for s, n in enumerate(lens):
            x = torch.randn((heads, n, d), generator=g) * (110.0 if fmt == E4M3 else 31.0)
            q = R.nearest(x.double(), fmt)
            bits = q.float().to(torch.float8_e4m3fn).view(torch.uint8) if fmt == E4M3 else q.to(torch.int8).view(torch.uint8)
            codes[s, :, :n] = bits.cuda()
            nb = -(-n // block)
            scales[s, :, :nb] = (torch.exp(spread * torch.randn((heads, nb), generator=g)) / (110.0 if fmt == E4M3 else 31.0)).cuda()
    return cache


def values(cache, s, n):
    """(k, v) of sequence s as float64 [h][n][d]."""
    fmt, block = cache.c.format, cache.c.block
    b = torch.arange(n) // block
    return tuple(R.decode(c[s, :, :n], fmt) * sc[s].cpu().double()[:, b, None]
                 for c, sc in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)))


def v_top(cache, s, n):
    """The largest V scale times the largest V code of a sequence."""
    scales = cache.v_scales[s, :, :-(-n // cache.c.block)].cpu().double()
    return float(scales.max() * R.decode(cache.v_codes[s, :, :n], cache.c.format).abs().max())


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("d,block,dtype", [(64, 16, F32), (64, 128, BF16), (128, 32, F16), (128, 128, BF16), (128, 64, F32)])
def test_append_is_bit_exact(fmt, d, block, dtype):
    # without rotation, codes and scales follow from IEEE operations alone: every one is equal; what is
    # behind the new tokens and what belongs to other blocks is untouched
    heads, max_ctx = 3, 300
    cache = T.Kv8Cache(heads, d, max_ctx, n_seqs=4, fmt=fmt, block=block)
    garbage(cache)
    want = [(R.decode(c, fmt), s.cpu().double()) for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales))]
    raw = cache.k_codes.cpu().clone(), cache.v_codes.cpu().clone()
    starts, lens, pos = [0, 0, 0, 7 * block % 200 // block * block], [250, 1, 129, 60], [0] * 4
    pos[3] = starts[3]
    step = 0
    while any(n > 0 for n in lens):  # calls of several sizes, so that blocks are started, filled and grown
        t = [130, 1, 7, 33, 1, 64][step % 6]
        counts = [min(t, n) for n in lens]
        size = 2.0 ** (step % 5)
        k, v = (normal((4, t, heads, d), 10 * step + i, size * (1 + i)).to(dtype) for i in range(2))
        cache.append(k.cuda(), v.cuda(), ints(*pos), counts=ints(*counts))
        for s in range(4):
            if counts[s]:
                for (codes, scales), x in zip(want, (k, v)):
                    R.store(x[s, :counts[s]], codes[s], scales[s], pos[s], fmt, block)
            pos[s] += counts[s]
            lens[s] -= counts[s]
        step += 1
    for (codes, scales), got, gs, was in zip(want, (cache.k_codes, cache.v_codes), (cache.k_scales, cache.v_scales), raw):
        for s in range(4):
            a, b = starts[s], pos[s]
            assert torch.equal(R.decode(got[s, :, a:b], fmt), codes[s, :, a:b]), s
            assert torch.equal(got[s, :, b:].cpu(), was[s, :, b:]), s  # rows behind the last token
            assert torch.equal(got[s, :, :a].cpu(), was[s, :, :a]), s
            assert torch.equal(gs[s].cpu().double().nan_to_num(-1), scales[s].nan_to_num(-1)), s


@pytest.mark.parametrize("fmt,d,theta,first", [(E4M3, 64, 500000.0, 0), (INT8, 128, 1e6, 77), (E4M3, 128, 10000.0, (1 << 24) - 40)])
def test_append_rotates_keys(fmt, d, theta, first):
    # a rotated key is off by a few fp32 roundings of its two terms and of its angle (together below
    # 2^-20 of their size); a code by that, in units of the scale, beside its own half step
    t, heads, block = 37, 2, 32
    buffers = None
    max_ctx = first + t if first < 1000 else 1 << 24
    cache = T.Kv8Cache(heads, d, max_ctx, fmt=fmt, block=block, buffers=buffers)
    k, v = normal((1, t, heads, d), 1).to(BF16), normal((1, t, heads, d), 2).to(BF16)
    cache.append(k.cuda(), v.cuda(), ints(first), rope_theta=theta)
    x = R.rotate(k[0].double(), first, theta)
    b0, b1 = first // block, (first + t - 1) // block
    got = R.decode(cache.k_codes[0, :, first:first + t], fmt).transpose(0, 1)
    scales = cache.k_scales[0, :, b0:b1 + 1].cpu().double()
    at = (first + torch.arange(t)) // block - b0
    for b in range(b1 - b0 + 1):
        amax = x[at == b].abs().amax(dim=(0, 2))
        if b > 0 or first % block == 0:
            assert (scales[:, b] * R.QMAX[fmt] / amax - 1).abs().max() < 2.0 ** -19
    s = scales[:, at].T[:, :, None]
    q = x / s
    far = R.half_step(q, fmt) * (1 + 2.0 ** -10) + 2.0 ** -19 * q.abs().amax() * 2
    assert bool(((got - q.clamp(-R.QMAX[fmt], R.QMAX[fmt])).abs() <= far).all())


def test_append_special_values():
    block, d = 16, 64
    cache = T.Kv8Cache(1, d, 96, fmt=E4M3, block=block)
    k = normal((1, 96, 1, d), 3)
    k[0, 0:16] = 0.0                 # a block of zeros
    k[0, 16:32] *= 1e-42             # subnormal values: the scale stops at 2^-126
    k[0, 40, 0, 5] = math.nan        # a NaN spoils its block alone
    k[0, 50, 0, 9] = -math.inf       # and so does an infinity
    k[0, 64:80] *= 1e37              # huge values
    v = k.flip(1).contiguous()
    cache.append(k.cuda(), v.cuda(), ints(0))
    s = cache.k_scales[0, 0].cpu()
    assert s[0] == 0 and s[1] == 2.0 ** -126 and math.isnan(s[2]) and math.isnan(s[3]) and torch.isfinite(s[4:]).all()
    for c in (cache.k_codes, cache.v_codes):  # no NaN code is ever written
        assert bool(((c & 0x7F) != 0x7F).all())
    kb, vb = cache.read(96, ints(0), dtype=F32)
    assert bool((kb[0, :16] == 0).all()) and bool(kb[0, 32:64].isnan().all())
    assert bool(kb[0, 64:].isfinite().all()) and bool(kb[0, 16:32].isfinite().all())
    # a block of zeros that grows takes its scale from the first values; a spoilt block stays so until it
    # is started again
    cache.append(torch.ones(1, 2, 1, d, device="cuda"), torch.ones(1, 2, 1, d, device="cuda"), ints(4))
    assert abs(float(cache.k_scales[0, 0, 0]) * 448 - 1) < 1e-6
    cache.append(torch.ones(1, 2, 1, d, device="cuda"), torch.ones(1, 2, 1, d, device="cuda"), ints(44))
    assert math.isnan(float(cache.k_scales[0, 0, 2]))
    cache.append(torch.ones(1, 2, 1, d, device="cuda"), torch.ones(1, 2, 1, d, device="cuda"), ints(32))
    assert float(cache.k_scales[0, 0, 2]) > 0


def test_positions_outside_the_cache_are_passed_over():
    cache = T.Kv8Cache(2, 64, 50, n_seqs=5)
    garbage(cache)
    was = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales)]
    x = torch.ones(5, 4, 2, 64, device="cuda")
    status = ints(0)
    pos, counts = ints(-1, 47, 50, 10, 2 ** 31 - 1), ints(4, 4, 1, 5, 4)
    cache.append(x, x, pos, counts=counts, status=status)
    assert int(status) == 1
    status.zero_()
    out = torch.full_like(x, 7.0)
    cache.read(4, pos, counts=counts, out=(out, out.clone()), status=status)
    assert int(status) == 1 and bool((out == 7).all())
    status.zero_()
    cache.attention(x, pos, counts=counts, out=out, status=status)
    assert int(status) == 1 and bool((out == 7).all())
    for t, w in zip((cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales), was):
        assert torch.equal(t.nan_to_num(-1) if t.is_floating_point() else t, w.nan_to_num(-1) if w.is_floating_point() else w)
    # one bad sequence among good ones; the status is cleared by a call without one
    cache.append(x, x, ints(0, 0, 99, 0, 0), status=status)
    assert int(status) == 1
    back = cache.read(4, ints(0, 0, 0, 0, 0), dtype=F32)[0]
    assert bool((back[[0, 1, 3, 4]] - 1).abs().max() < 2.0 ** -4)
    cache.append(x, x, ints(0, 0, 0, 0, 0), status=status)
    assert int(status) == 0


def test_strided_rows_and_the_bf16_cache_layout():
    # one layer of a bf16 cache [h][ctx][d] as rows, and k and v inside one fused projection buffer
    heads, d, n = 3, 64, 70
    layer = normal((heads, 90, d), 5).to(BF16).cuda()
    rows = layer.transpose(0, 1)[None, :n]
    fused = torch.zeros(1, n, (heads * 2 + 2) * d, dtype=BF16, device="cuda")
    fused[0, :, 2 * d:2 * d + heads * d] = rows[0].reshape(n, -1)
    fused[0, :, 2 * d + heads * d:] = (rows[0] * 2).reshape(n, -1)
    k = fused[..., 2 * d:2 * d + heads * d].view(1, n, heads, d)
    v = fused[..., 2 * d + heads * d:].view(1, n, heads, d)
    a, b = T.Kv8Cache(heads, d, 90), T.Kv8Cache(heads, d, 90)
    a.append(rows, rows * 2, ints(3))
    b.append(k, v, ints(3))
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_codes, b.v_codes) and torch.equal(a.v_scales, b.v_scales)
    back = torch.full((2, heads, 90, d), 9.0, dtype=BF16, device="cuda")
    views = [back[i].transpose(0, 1)[None, 10:10 + n] for i in range(2)]
    a.read(n, ints(3), out=views)
    ref = a.read(n, ints(3))
    assert torch.equal(views[0], ref[0]) and torch.equal(views[1], ref[1])
    assert bool((back[:, :, :10] == 9).all()) and bool((back[:, :, 10 + n:] == 9).all())


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("d,dtype", [(64, F32), (128, BF16), (64, F16)])
def test_read_is_exact(fmt, d, dtype):
    cache = filled(2, d, [100, 37, 1], 100, fmt, 16, seed=4)
    pos, counts = [3, 30, 0], [97, 7, 1]
    out = tuple(torch.full((3, 97, 2, d), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    cache.read(97, ints(*pos), counts=ints(*counts), out=out)
    for s in range(3):
        k, v = values(cache, s, pos[s] + counts[s])
        for got, x in zip(out, (k, v)):
            # code * scale has at most 31 significant bits: fp32's rounding, then the dtype's
            want = x[:, pos[s]:].transpose(0, 1).float().to(dtype)
            assert torch.equal(got[s, :counts[s]].cpu(), want)
            assert bool((got[s, counts[s]:] == 5).all())


def test_growing_token_by_token_stays_within_two_steps():
    # tokens of rising size: the scale at least doubles each time it grows, so the held codes' errors are
    # half steps of a geometric series: below 1/2 + 1/2 (1 + 1/2 + ...) = 1.5 steps of the final scale
    d, n = 64, 64
    x = torch.linspace(0.01, 3.0, n)[None, :, None, None] * normal((1, n, 2, d), 6).clamp(-2, 2)
    cache = T.Kv8Cache(2, d, n, fmt=INT8, block=64)
    for i in range(n):
        cache.append(x[:, i:i + 1].cuda(), x[:, i:i + 1].cuda(), ints(i))
    k, v = cache.read(n, ints(0), dtype=F32)
    step = cache.k_scales.cpu()[0, :, 0][None, :, None]
    assert bool(((k[0].cpu() - x[0]).abs() <= 1.5 * step * (1 + 1e-5)).all())
    assert torch.equal(k, v)


# ------------------------------------------------------------------ attention

def check_attention(cache, lens, counts, hq, dtype, theta, q_scale=1.0, seed=0, t=None, lse=True):
    hk, d = cache.n_kv_heads, cache.head_dim
    n_seqs, t = len(lens), t or max(counts)
    pos = [n - c for n, c in zip(lens, counts)]
    q = normal((n_seqs, t, hq, d), 100 + seed, q_scale).to(dtype)
    out = torch.full((n_seqs, t, hq, d), 3.0, dtype=dtype, device="cuda")
    sums = torch.full((n_seqs, t, hq), 3.0, device="cuda")
    status = ints(0)
    cache.attention(q.cuda(), ints(*pos), counts=ints(*counts), rope_theta=theta, out=out, lse=sums if lse else None, status=status)
    assert int(status) == 0
    worst = 0.0
    for s in range(n_seqs):
        c, n = counts[s], lens[s]
        assert bool((out[s, c:] == 3).all()) and bool((sums[s, c:] == 3).all())  # rows past the count
        if c == 0:
            continue
        k, v = values(cache, s, n)
        want, ls, size, mean = R.attend(R.rotate(q[s, :c].double(), pos[s], theta), k, v, pos[s])
        far, far_lse = R.attend_bounds(want, size, mean, d, n, dtype, v_top(cache, s, n))
        got = out[s, :c].cpu().double()
        assert bool(got.isfinite().all()), s
        err = ((got - want).abs() / far).max()
        worst = max(worst, float(err))
        assert float(err) <= 1, (s, float(err))
        if lse:
            e = ((sums[s, :c].cpu().double() - ls).abs() / (far_lse + ls.abs() * 2.0 ** -22)).max()
            assert float(e) <= 1, (s, float(e))
    return worst


HEADS = [(4, 2, 64), (32, 8, 64), (12, 2, 128), (8, 1, 64), (3, 3, 128), (40, 8, 64), (16, 1, 128), (17, 1, 64)]


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("dtype", [BF16, F32, F16])
def test_attention_single_tokens(hq, hk, d, dtype):
    fmt = E4M3 if hq % 3 else INT8
    lens = [1, 2, 31, 32, 33, 63, 64, 65, 127, 200, 1000]
    cache = filled(hk, d, lens, 1003, fmt, 16, seed=hq)
    check_attention(cache, lens, [1] * len(lens), hq, dtype, 10000.0, seed=d)


def test_one_workspace_serves_every_call_of_a_small_cache():
    cache = filled(1, 64, [9], 9, E4M3, 16, seed=1)
    for t in (1, 2, 9):
        check_attention(cache, [9], [t], 40, F32, 10000.0)
    assert cache.workspace_bytes(1, 1) == cache.workspace_bytes(40, 9)


@pytest.mark.parametrize("fmt,block", [(E4M3, 16), (E4M3, 32), (INT8, 64), (INT8, 128), (E4M3, 128)])
@pytest.mark.parametrize("hq,hk,d", [(32, 4, 64), (12, 2, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_several_tokens_ragged(fmt, block, hq, hk, d, dtype):
    lens, counts = [8, 5, 70, 131, 500, 64, 9], [8, 1, 3, 8, 7, 0, 2]
    cache = filled(hk, d, lens, 501, fmt, block, seed=block)
    check_attention(cache, lens, counts, hq, dtype, 500000.0, t=8)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (12, 2, 128), (32, 4, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32, F16])
@pytest.mark.parametrize("lens,counts", [([100], [100]), ([300, 190], [130, 190]), ([257], [97]), ([129, 40, 1], [128, 1, 1])])
def test_attention_prompts(hq, hk, d, dtype, lens, counts):
    cache = filled(hk, d, lens, max(lens), INT8 if hq == 12 else E4M3, 64, seed=len(lens))
    check_attention(cache, lens, counts, hq, dtype, 10000.0)


@pytest.mark.parametrize("hq,hk,d,n,t,fmt", [(32, 8, 64, 8192, 512, E4M3), (12, 2, 128, 8192, 512, INT8), (4, 4, 64, 5000, 300, INT8),
                                             (16, 1, 128, 6001, 77, E4M3), (12, 2, 128, 2048, 2048, INT8), (16, 2, 64, 9000, 16, INT8)])
def test_long_prompts_whose_maxima_keep_rising(hq, hk, d, n, t, fmt):
    # keys grow along the context, so that running maxima rise and outputs are rescaled far into a run of key
    # tiles; the outcome is the same every time and within the bounds
    k = normal((1, n, hk, d), 1) * torch.linspace(0.2, 4, n)[None, :, None, None]
    v = normal((1, n, hk, d), 2)
    cache = T.Kv8Cache(hk, d, n, fmt=fmt, block=64)
    cache.append(k.cuda(), v.cuda(), ints(0))
    q = normal((1, t, hq, d), 3, 1.5).to(BF16)
    outs = [cache.attention(q.cuda(), ints(n - t)) for _ in range(20)]
    assert all(torch.equal(o, outs[0]) for o in outs)
    kk, vv = values(cache, 0, n)
    for a in range(0, t, 128):
        b = min(t, a + 128)
        want, _, size, mean = R.attend(q[0, a:b].double(), kk[:, :n - t + b], vv[:, :n - t + b], n - t + a)
        far, _ = R.attend_bounds(want, size, mean, d, n, BF16, v_top(cache, 0, n))
        assert bool(((outs[0][0, a:b].cpu().double() - want).abs() <= far).all()), a
        # most elements are far nearer than the worst case: within a few roundings of the row's size
        rms = want.square().mean().sqrt()
        assert float((outs[0][0, a:b].cpu().double() - want).abs().max() / rms) < 0.1, a


def test_prompts_of_a_ragged_batch():
    lens, counts = [700, 64, 1300, 5, 0, 333], [300, 64, 513, 5, 0, 1]
    lens[4] = 1  # nothing new there
    for hq, hk, d in ((6, 2, 64), (8, 8, 128), (10, 1, 64)):
        cache = filled(hk, d, lens, 1300, E4M3, 32, seed=hq, spread=0.3)
        check_attention(cache, lens, counts, hq, BF16, 500000.0, t=520)


@pytest.mark.parametrize("hq,hk,d", [(8, 8, 64), (6, 6, 128), (24, 8, 64)])
def test_prompts_of_one_and_of_two_row_tiles_in_turn(hq, hk, d):
    # more units of work than multiprocessors, so that one takes a unit of up to 128 query rows and then a larger one
    lens = [700 + 37 * (s % 5) for s in range(64)]
    counts = [(70, 200, 128, 129, 66)[s % 5] for s in range(64)]
    cache = filled(hk, d, lens, max(lens), E4M3, 64, seed=hq, spread=0.3)
    check_attention(cache, lens, counts, hq, BF16, 0.0, t=200)
    check_attention(cache, lens, counts[::-1], hq, BF16, 10000.0, t=200)


@pytest.mark.parametrize("hq,hk,d,n,dtype", [(12, 2, 128, 40000, F32), (32, 8, 64, 9001, BF16), (4, 2, 64, 70000, BF16)])
def test_attention_long_context_is_split_and_joined(hq, hk, d, n, dtype):
    cache = filled(hk, d, [n], n + 7, E4M3, 128, seed=9)
    check_attention(cache, [n], [1], hq, dtype, 1e6)


def test_attention_offsets_past_32_bits():
    # 2.1 and 4.3 GB of codes lie before the sequences read here
    n_seqs, heads, d, ctx = 3, 2, 64, (1 << 24)
    cache = T.Kv8Cache(heads, d, ctx, n_seqs=n_seqs, block=128)
    pos = [ctx - 300, ctx - 300, ctx - 300]
    x, y = normal((n_seqs, 300, heads, d), 1).to(BF16), normal((n_seqs, 300, heads, d), 2).to(BF16)
    cache.append(x.cuda(), y.cuda(), ints(*pos))
    back = cache.read(300, ints(*pos), dtype=F32)
    assert float((back[0].cpu() - x.float()).abs().max()) < 4 * 2.0 ** -4
    assert float((back[1].cpu() - y.float()).abs().max()) < 4 * 2.0 ** -4
    # all earlier keys and values are zero (scale 0): a score 0 each, and the last ones with larger scores
    q = normal((n_seqs, 1, 4, d), 3)
    out = cache.attention(q.cuda(), ints(*[ctx - 1] * n_seqs))
    for s in range(n_seqs):
        k, v = back[0][s].cpu().double().transpose(0, 1), back[1][s].cpu().double().transpose(0, 1)
        for h in range(4):
            e = torch.exp((k[h // 2] @ q[s, 0, h].double()) / 8.0)
            want = (e @ v[h // 2]) / (e.sum() + ctx - 300)
            # 2^24 equal weights add up in parts of at most 2^17 keys: the sum is off by 2^-7 at most
            assert float((out[s, 0, h].cpu().double() - want).abs().max()) <= 2.0 ** -6 * float(want.abs().max())


@pytest.mark.parametrize("q_scale", [1e-30, 1e-3, 30.0, 1e4])
def test_attention_query_sizes(q_scale):
    # tiny queries (uniform weights) to huge ones (one key takes all): the scores' bound grows with them, so
    # for the huge ones the keys are the cache's own first key and its negative, scores far apart
    cache = filled(2, 64, [500], 500, E4M3, 64, seed=2, spread=0.2)
    if q_scale <= 30:
        check_attention(cache, [500], [1], 8, F32, 0.0, q_scale=q_scale)
        return
    q = torch.full((1, 1, 8, 64), q_scale)
    out = cache.attention(q.cuda(), ints(499))
    k, v = values(cache, 0, 500)
    want, _, _, _ = R.attend(q[0].double(), k, v, 499)
    s = (k.sum(-1) * q_scale / 8).sort(dim=1, descending=True).values
    assert bool((s[:, 0] - s[:, 1] > 100).all())  # the largest score leads by far: its value is the answer
    assert float((out[0].cpu().double() - want).abs().max()) <= 1e-5 * float(want.abs().max())


@pytest.mark.parametrize("t,dtype", [(1, F32), (5, BF16), (150, BF16)])
def test_queries_near_the_types_end(t, dtype):
    # as large as the type holds, against keys as small: ordinary scores. The scales fall below 2^-126 and lose bits
    # themselves (steps of 2^-149 at 2^-127), so the formula over the cache as it then is says what is right
    cache = filled(2, 64, [400], 400, E4M3, 64, seed=12, spread=0.2)
    q = normal((1, t, 8, 64), 13).clamp(-3, 3).to(dtype)
    cache.k_scales.mul_(2.0 ** -120)
    got = cache.attention((q * 2.0 ** 120).cuda(), ints(400 - t))[0].cpu().double()
    k, v = values(cache, 0, 400)
    want, _, size, mean = R.attend(q[0].double() * 2.0 ** 120, k, v, 400 - t)
    far, _ = R.attend_bounds(want, size, mean, 64, 400, dtype, v_top(cache, 0, 400))
    assert bool((size < 100).all()) and bool(got.isfinite().all()) and bool(((got - want).abs() <= far).all())


@pytest.mark.parametrize("t,dtype", [(1, F32), (1, BF16), (5, BF16), (40, F32), (150, BF16)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (2, 1, 128)])
@pytest.mark.parametrize("down", [110, 120, 125])
def test_queries_near_zero_against_huge_keys(hq, hk, d, t, dtype, down):
    # as small as normal numbers get, against keys as large: ordinary scores
    cache = filled(hk, d, [400], 400, E4M3, 64, seed=12, spread=0.2)
    q = normal((1, t, hq, d), 13).clamp(-3, 3).to(dtype).float().mul(2.0 ** -down).to(dtype)
    cache.k_scales.mul_(2.0 ** down)
    got = cache.attention(q.cuda(), ints(400 - t))[0].cpu().double()
    k, v = values(cache, 0, 400)
    want, _, size, mean = R.attend(q[0].double(), k, v, 400 - t)
    far, _ = R.attend_bounds(want, size, mean, d, 400, dtype, v_top(cache, 0, 400))
    assert bool((size < 100).all()) and bool(got.isfinite().all()) and bool(((got - want).abs() <= far).all())

@pytest.mark.parametrize("hq,hk,d", [(10, 2, 64), (6, 1, 128)])
def test_fp32_rows_keep_their_precision_over_many_keys(hq, hk, d):
    # sums that were cut off at each step would be off by half a step (2^-24) for each of the 200 or more products of 16
    # keys in a warp's run, one way; rounded sums of tiles stay within a few steps: rms below 2^-20 of the outputs' rms
    n, seqs = 8000, 40
    cache = T.Kv8Cache(hk, d, n, n_seqs=seqs)
    k, v = (normal((1, n, hk, d), i).expand(seqs, n, hk, d).cuda() for i in (1, 2))
    cache.append(k, v, ints(*[0] * seqs))
    q = normal((seqs, 1, hq, d), 3)
    out = cache.attention(q.cuda(), ints(*[n - 1] * seqs))
    kk, vv = values(cache, 0, n)
    for s in (0, 17, 39):
        want, _, _, _ = R.attend(q[s].double(), kk, vv, n - 1)
        assert float((out[s].cpu().double() - want).square().mean().sqrt() / want.square().mean().sqrt()) <= 2.0 ** -20


def test_attention_scales_far_apart():
    # V blocks whose scales span 2^-40 .. 2^40, a block of zeros, one of the smallest scale
    cache = filled(2, 64, [320], 320, INT8, 32, seed=8)
    cache.v_scales[0, :, :10] = (2.0 ** torch.linspace(-40, 40, 10)).cuda()
    cache.v_scales[0, 0, 4] = 0.0
    cache.v_scales[0, 1, 9] = 2.0 ** -126
    check_attention(cache, [320], [1], 6, F32, 10000.0)
    check_attention(cache, [320], [9], 6, F32, 10000.0)
    cache.k_scales[0, :, 3] = 0.0
    check_attention(cache, [320], [200], 6, BF16, 10000.0)


@pytest.mark.parametrize("dtype,t", [(F32, 1), (BF16, 1), (F32, 40), (BF16, 40), (BF16, 100)])
@pytest.mark.parametrize("far", [45, 70, 110])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (2, 1, 128)])
def test_blocks_of_zeros_count_beside_blocks_of_huge_values(hq, hk, d, far, dtype, t):
    # a key whose values are zero has its weight in the softmax whatever the V scales of other keys are: zero and huge
    # blocks within one tile of keys, and in both orders across tiles
    n, block = 640, 16
    zeros, huge = 0.0, 2.0 ** far
    for row in ([zeros, huge] * 20, [zeros] * 20 + [huge] * 20, [huge] * 20 + [zeros] * 20, [zeros] * 39 + [huge],
                [huge] + [zeros] * 39, [2.0 ** -60, huge, 2.0 ** -126, zeros] * 10):
        cache = filled(hk, d, [n], n, INT8, block, seed=far)
        cache.v_scales[0, :, :n // block] = torch.tensor(row, device="cuda")
        check_attention(cache, [n], [t], hq, dtype, 10000.0)


@pytest.mark.parametrize("dtype,t,n", [(F32, 1, 30000), (BF16, 1, 30000), (BF16, 60, 9200)])
def test_parts_of_zeros_and_of_huge_values_are_joined(dtype, t, n):
    # runs of keys in several warps and multiprocessors, some with zeros alone and some with huge values
    for row in (torch.arange(n // 100) % 7 < 3, torch.arange(n // 100) < n // 150, torch.arange(n // 100) >= n // 150):
        cache = filled(2, 64, [n], n, INT8, 16, seed=n)
        cache.v_scales[0] = torch.where(row[torch.arange(n // 16) * 16 // 100], 0.0, 2.0 ** 100).cuda()[None]
        check_attention(cache, [n], [t], 8, dtype, 0.0)


@pytest.mark.parametrize("dtype,t", [(F32, 40), (BF16, 20), (BF16, 100)])
def test_huge_values_that_a_row_does_not_see_leave_it_alone(dtype, t):
    # the last block is huge: rows before it have the bits that they have with an ordinary block there
    n = 200
    cache = filled(2, 64, [n], n, INT8, 16, seed=5)
    q = normal((1, t, 8, 64), 6).to(dtype).cuda()
    want = cache.attention(q, ints(n - t))[:, :t - 8].cpu().double()
    cache.v_scales[0, :, 192 // 16:] = 2.0 ** 115
    got = cache.attention(q, ints(n - t))[:, :t - 8].cpu().double()
    far = 2.0 ** -7 if dtype == BF16 else 2.0 ** -16  # (sums in another order: a few roundings of the type)
    assert bool(((got - want).abs() <= far * want.abs().amax(dim=-1, keepdim=True)).all())

@pytest.mark.parametrize("t,d", [(1, 64), (100, 64), (1, 128), (100, 128)])
@pytest.mark.parametrize("below", [20.3, 22.4, 25.55, 28.7, 30.6, 33.4])
def test_many_keys_far_below_the_leading_one(below, t, d):
    # the first key has all but n 2^-below of the weight and values of 0: what comes out is the tail's sum, whose
    # weights are held to 2^-39 of the largest
    n = 600
    cache = T.Kv8Cache(1, d, n, block=16)
    k, v = torch.zeros(1, n, 1, d), torch.ones(1, n, 1, d)
    k[0, 0], v[0, 0] = 1.0, 0.0
    cache.append(k.cuda(), v.cuda(), ints(0))
    cache.k_scales[0, 0, 0] = below / math.log2(math.e) / math.sqrt(d) / 448
    q = torch.ones(1, t, 2, d)
    got = cache.attention(q.to(BF16).cuda(), ints(n - t))[0].cpu().double()
    kk, vv = values(cache, 0, n)
    want, _, size, mean = R.attend(q[0].double(), kk, vv, n - t)
    far, _ = R.attend_bounds(want, size, mean, d, n, BF16, v_top(cache, 0, n))
    assert bool(((got - want).abs() <= far).all()), float((got / want - 1).abs().max())

@pytest.mark.parametrize("t,dtype", [(1, F32), (1, BF16), (40, F32), (5, BF16), (100, BF16)])
@pytest.mark.parametrize("fmt", [INT8, E4M3])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (2, 1, 128)])
def test_values_near_the_types_end(hq, hk, d, fmt, t, dtype):
    # blocks begun with almost the largest numbers and grown by the largest: V scales of up to 2^122
    n = 320
    cache = T.Kv8Cache(hk, d, n, fmt=fmt, block=32)
    k, v = normal((1, n, hk, d), 1), torch.rand((1, n, hk, d), generator=torch.Generator().manual_seed(2)) * 2 - 1
    v *= 3.2e38
    v[0, 0::32, :, 3], v[0, 31::32, :, 3] = 3.39e38, 3.4028e38
    for a in range(0, n, 32):
        for b, e in ((a, a + 31), (a + 31, a + 32)):
            cache.append(k[:, b:e].cuda(), v[:, b:e].cuda(), ints(b))
    if fmt == INT8:
        assert float(cache.v_scales.max()) > 2.0 ** 122
    check_attention(cache, [n], [t], hq, dtype, 10000.0)

@pytest.mark.parametrize("dtype,t", [(F32, 40), (BF16, 40), (BF16, 150)])
def test_a_spoilt_block_reaches_the_rows_that_see_it_alone(dtype, t):
    block, n = 16, 200
    for which in ("k_scales", "v_scales"):
        cache = filled(1, 64, [n], n, E4M3, block, seed=3)
        getattr(cache, which)[0, 0, 11] = math.nan  # positions 176 .. 191
        q = normal((1, t, 4, 64), 4).to(dtype)
        out = cache.attention(q.cuda(), ints(n - t))
        seen = (torch.arange(n - t, n) >= 176).tolist()
        for i in range(t):
            assert bool(out[0, i].isnan().all()) == seen[i] and bool(out[0, i].isfinite().all()) != seen[i], i


def test_a_query_that_is_not_finite_spoils_its_own_row():
    cache = filled(2, 64, [100], 100, E4M3, 64, seed=3)
    q = normal((1, 6, 8, 64), 4)
    q[0, 2, 3, 7] = math.nan
    q[0, 4, 1, 0] = math.inf
    out = cache.attention(q.cuda(), ints(94))
    bad = torch.zeros(6, 8, dtype=torch.bool)
    bad[2, 3] = bad[4, 1] = True
    assert torch.equal(out[0].isnan().all(-1).cpu(), bad) and torch.equal(out[0].isnan().any(-1).cpu(), bad)


def test_out_may_be_the_queries_memory():
    cache = filled(2, 64, [3000, 40], 3000, E4M3, 64, seed=5)
    q = normal((2, 9, 8, 64), 6).to(BF16).cuda()
    want = cache.attention(q, ints(2991, 31))
    got = cache.attention(q, ints(2991, 31), out=q)
    assert got is q and torch.equal(got, want)


def test_results_do_not_depend_on_timing_or_neighbours():
    cache = filled(2, 128, [5000, 1, 700], 5000, INT8, 64, seed=7)
    q = normal((3, 2, 12, 128), 8).to(BF16).cuda()
    pos, counts = ints(4998, 0, 698), ints(2, 1, 2)
    want = cache.attention(q, pos, counts=counts)
    for _ in range(20):
        assert torch.equal(cache.attention(q, pos, counts=counts), want)


def test_two_streams_with_workspaces_of_their_own():
    cache = filled(2, 64, [20000], 20000, E4M3, 64, seed=7)
    qs = [normal((1, 1, 8, 64), 20 + i).to(BF16).cuda() for i in range(2)]
    want = [cache.attention(q, ints(19999)) for q in qs]
    pos = ints(19999)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(cache.workspace_bytes(8, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cache.attention(qs[i], pos, workspace=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_results_made_for_another_stream_belong_to_it():
    # the current stream is busy: what it fills later must not reach results that the other stream has written
    cache = filled(2, 64, [700], 700, E4M3, 64, seed=7)
    q = normal((1, 3, 8, 64), 20).to(BF16).cuda()
    x, t = normal((5, 1000), 21).cuda(), ints(1, 2, 3, 4, 5)
    pos, zero = ints(697), ints(0)
    want = (cache.attention(q, pos), *cache.read(700, zero), *T.logprobs(x, t, 4))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        torch.cuda._sleep(20_000_000)
        got = (cache.attention(q, pos, stream=handle), *cache.read(700, zero, stream=handle), *T.logprobs(x, t, 4, stream=handle))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_from_several_host_threads():
    import threading
    caches = [filled(1, 64, [50] * n, 50, E4M3, 64, seed=n) for n in (1, 40, 700)]
    qs = [normal((c.n_seqs, 1, 2, 64), 30).cuda() for c in caches]
    poss = [ints(*[49] * c.n_seqs) for c in caches]
    want = [c.attention(q, p) for c, q, p in zip(caches, qs, poss)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        stream = torch.cuda.Stream()
        for _ in range(200):
            try:
                out = caches[i].attention(qs[i], poss[i], stream=stream)
            except T.TinferError as e:
                wrong.append(e)
                return
            stream.synchronize()
            if not torch.equal(out, want[i]):
                wrong.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_strides_of_single_extents_do_not_matter():
    cache = filled(2, 64, [90], 90, E4M3, 64, seed=7)
    q = normal((1, 1, 8, 64), 20).to(BF16).cuda()
    odd = torch.as_strided(q, q.shape, (7, 3, 64, 1))
    assert torch.equal(cache.attention(odd, ints(89)), cache.attention(q, ints(89)))


def test_captured_step_follows_the_positions():
    heads, hq, d, n = 2, 8, 64, 40
    k, v, q = (normal((n, 1, 1, h, d), i).to(BF16).cuda() for i, h in enumerate((heads, heads, hq)))
    a, b = T.Kv8Cache(heads, d, n), T.Kv8Cache(heads, d, n)
    pos, kk, vv, qq = ints(0), k[0].clone(), v[0].clone(), q[0].clone()
    out = torch.zeros_like(qq)

    def step(c):
        c.append(kk, vv, pos, rope_theta=10000.0)
        c.attention(qq, pos, rope_theta=10000.0, out=out)
        pos.add_(1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    pos.zero_()
    for i in range(n):
        for dst, src in ((kk, k), (vv, v), (qq, q)):
            dst.copy_(src[i])
        graph.replay()
        got = out.clone()
        b.append(k[i], v[i], ints(i), rope_theta=10000.0)
        assert torch.equal(got, b.attention(q[i], ints(i), rope_theta=10000.0)), i
    assert torch.equal(a.k_codes, b.k_codes) and torch.equal(a.v_scales, b.v_scales) and int(pos) == n


def test_prompt_then_tokens_equals_what_the_cache_holds():
    # the run of a serving program: projections of a prompt by the prefill product, stored as they come out
    # (fp32, fused buffer), attention over the prompt, then single and drafted tokens
    hq, hk, d, hidden, n = 4, 2, 64, 256, 75
    x = synth.normal_bf16("kv8.x", (n + 9, hidden), 0.0, 1.0, 0)
    w = synth.normal_bf16("kv8.w", ((hq + 2 * hk) * d, hidden), 0.0, 0.06, 0)
    xd, wd = (torch.from_numpy(a.view(np.int16)).cuda() for a in (x, w))
    y = torch.empty((n + 9, w.shape[0]), device="cuda")
    assert T.tinfer_op_gemm_bf16(n + 9, w.shape[0], hidden, xd, wd, y) == T.TINFER_OK
    rows = y[None]
    q = rows[..., :hq * d].view(1, n + 9, hq, d)
    k = rows[..., hq * d:(hq + hk) * d].view(1, n + 9, hk, d)
    v = rows[..., (hq + hk) * d:].view(1, n + 9, hk, d)
    cache = T.Kv8Cache(hk, d, 128, block=32)
    outs, at = [], 0
    for t in (n, 1, 1, 1, 6):
        cache.append(k[:, at:at + t], v[:, at:at + t], ints(at), rope_theta=10000.0)
        got = cache.attention(q[:, at:at + t], ints(at), rope_theta=10000.0)
        kk, vv = values(cache, 0, at + t)
        want, _, size, mean = R.attend(R.rotate(q[0, at:at + t].cpu().double(), at, 10000.0), kk, vv, at)
        far, _ = R.attend_bounds(want, size, mean, d, at + t, F32, v_top(cache, 0, at + t))
        assert bool(((got[0].cpu().double() - want).abs() <= far).all()), t
        outs.append(got)
        at += t
    # and what the cache holds is near what was stored: e4m3 rounds by 2^-4 of a value, or 2^-10 of the scale
    back = cache.read(n, ints(0), dtype=F32)[1][0].cpu().double()
    ref = v[0, :n].cpu().double()
    top = ref.view(n, hk, d)
    block_top = torch.stack([top[b:b + 32].abs().amax(dim=(0, 2)) for b in range(0, n, 32)])
    far = ref.abs() * 2.0 ** -4 * (1 + 1e-6) + (2 * block_top / 448 * 2.0 ** -10)[torch.arange(n) // 32][:, :, None]
    # a block grown by later tokens rounds its subnormals again, in units of at most twice the largest / 448
    later = cache.v_scales[0].cpu().double().T[torch.arange(n) // 32][:, :, None] * 2.0 ** -9
    assert bool(((back - ref).abs() <= far + later).all())


def test_a_prefix_kept_in_8_bits_goes_back_to_the_engine():
    # the engine's bf16 cache stored in 8 bits layer by layer and read back: the step that follows is bit for bit
    # the step over the values that the 8-bit cache stands for
    cfg = synth.config("tiny", max_ctx=64)
    w = synth.make_model(cfg, seed=0)
    K, V = synth.make_kv(cfg, 40)
    a = T.Engine(cfg, w, T.TINFER_MEGAKERNEL, kv=(K, V))
    b = T.Engine(cfg, w, T.TINFER_MEGAKERNEL, kv=(K, V))
    for layer in range(cfg["n_layers"]):
        cache = T.Kv8Cache(cfg["n_kv_heads"], cfg["head_dim"], 40, fmt=INT8, block=16)
        ka, va = (t[layer].view(BF16).transpose(0, 1)[None, :40] for t in (a.k, a.v))
        cache.append(ka, va, ints(0))
        kv = values(cache, 0, 40)
        cache.read(40, ints(0), out=(ka, va))
        for eng_t, x in zip((b.k, b.v), kv):
            eng_t[layer, :, :40] = x.float().to(BF16).view(torch.int16).cuda()
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    for eng in (a, b):
        eng.step(5, 40)
    torch.cuda.synchronize()
    assert a.error() == T.TINFER_OK and b.error() == T.TINFER_OK
    assert torch.equal(a.logits, b.logits) and bool(a.logits.isfinite().all())
    a.close()
    b.close()


@pytest.mark.parametrize("hq,hk,d,t,dtype", [(8, 2, 64, 1, BF16), (32, 8, 64, 5, F32), (12, 2, 128, 1, F16), (8, 2, 64, 200, BF16),
                                             (12, 2, 128, 300, BF16), (8, 8, 64, 64, BF16)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(hq, hk, d, t, dtype):
    # one arrival of each pipeline stays away (every copy and product completes): the kernel gives up after 5 ms, issues
    # nothing more and ends. Runs are tens of tiles long, and a limit for each of them would take seconds
    import time
    n = 40000
    cache = filled(hk, d, [n], n, E4M3, 64, seed=3)
    q = normal((1, t, hq, d), 4).to(dtype).cuda()
    pos, status = ints(n - t), ints(0)
    want = cache.attention(q, pos, status=status)
    assert int(status) == 0
    cache.c.format |= T.TINFER_KV8_DEBUG_WITHHOLD
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    cache.attention(q, pos, out=out, status=status)
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert int(status) == 2 and took < 0.5, took
    cache.c.format &= ~T.TINFER_KV8_DEBUG_WITHHOLD
    assert torch.equal(cache.attention(q, pos, status=status), want) and int(status) == 0

def test_the_cache_gathers_what_calls_without_a_status_report():
    cache = filled(2, 64, [500], 500, E4M3, 64, seed=3)
    q, x = normal((1, 3, 8, 64), 4).cuda(), normal((1, 3, 2, 64), 5).cuda()
    assert cache.error() == 0
    cache.attention(q, ints(498))  # past the end
    cache.attention(q, ints(400))  # a good call does not clear it
    assert cache.error() == 1 and cache.error() == 0
    cache.append(x, x, ints(-1))
    status = ints(7)
    cache.append(x, x, ints(0), status=status)
    assert int(status) == 0 and cache.error() == 1
    cache.read(3, ints(499), status=status)
    assert int(status) == 1 and cache.error() == 0
    cache._kept.format |= T.TINFER_KV8_DEBUG_WITHHOLD
    cache.attention(q, ints(400))
    cache._kept.format &= ~T.TINFER_KV8_DEBUG_WITHHOLD
    cache.read(3, ints(499))
    assert cache.error() == 3 and cache.error() == 0
    assert cache.attention(q, ints(400)).isfinite().all() and cache.error() == 0

def test_a_cache_over_given_buffers_is_ready_for_any_stream():
    a = filled(2, 64, [300], 300, E4M3, 64, seed=3)
    q, pos, s = normal((1, 3, 8, 64), 4).cuda(), ints(299), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    tmp = torch.empty(a.workspace_bytes(), dtype=torch.uint8, device="cuda").fill_(7)
    del tmp  # its memory may be the workspace's, and the fill is yet to come
    b = T.Kv8Cache(2, 64, 300, buffers=(a.k_codes, a.v_codes, a.k_scales, a.v_scales))
    assert torch.cuda.current_stream().query()
    b.attention(q, pos, stream=s)  # past the end: reported
    torch.cuda.synchronize()
    assert b.error() == 1

def time_of(call, n=5):
    for _ in range(3):
        call()
    times = []
    for _ in range(9):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) / n)
    return sorted(times)[4]


@pytest.mark.parametrize("hq,hk,d", [(32, 8, 64), (12, 2, 128)])
def test_one_long_sequence_beside_single_tokens_is_dealt_out_evenly(hq, hk, d):
    # a prompt's chunk and 31 decode steps in one call: no longer than a few times the two calls by themselves, and right
    n, t, seqs = 2000, 256, 32
    cache = filled(hk, d, [n + t] * seqs, n + t, E4M3, 64, seed=6, spread=0.3)
    counts = [t] + [1] * (seqs - 1)
    check_attention(cache, [n + c for c in counts], counts, hq, F32, 0.0)
    q, pos = normal((seqs, t, hq, d), 7).cuda(), ints(*[n] * seqs)
    out = torch.zeros_like(q)
    mixed = time_of(lambda: cache.attention(q, pos, counts=ints(*counts), out=out))
    chunk = time_of(lambda: cache.attention(q, pos, counts=ints(t, *[0] * (seqs - 1)), out=out))
    step = time_of(lambda: cache.attention(q, pos, counts=ints(*[1] * seqs), out=out))
    assert mixed < 2.5 * (chunk + step), (mixed, chunk, step)

@pytest.mark.parametrize("t,dtype", [(1, F32), (40, F32), (40, BF16), (100, BF16)])
def test_a_call_without_any_new_token_does_nothing(t, dtype):
    for seqs in (1, 40):
        cache = filled(2, 64, [200] * seqs, 200, E4M3, 64, seed=3)
        q, status = normal((seqs, t, 8, 64), 4).to(dtype).cuda(), ints(0)
        out, lse = torch.full_like(q, 5.0), torch.full((seqs, t, 8), 5.0, device="cuda")
        for pos, counts, bits in (([0] * seqs, [0] * seqs, 0), ([200] * seqs, [0] * seqs, 0), ([-1] * seqs, [t] * seqs, 1)):
            cache.attention(q, ints(*pos), counts=ints(*counts), out=out, lse=lse, status=status)
            assert int(status) == bits and bool((out == 5).all()) and bool((lse == 5).all())

@pytest.mark.parametrize("hq,hk,d,t,dtype", [(8, 2, 64, 150, BF16), (12, 2, 128, 80, BF16), (8, 2, 64, 12, F32), (8, 2, 64, 70, F16)])
def test_two_captured_calls_replayed_side_by_side_follow_their_inputs(hq, hk, d, t, dtype):
    n, seqs = 900, 5
    cache = filled(hk, d, [n] * seqs, n, INT8, 32, seed=3)
    ws = [torch.empty(cache.workspace_bytes(), dtype=torch.uint8, device="cuda") for _ in range(2)]
    qs = [torch.zeros(seqs, t, hq, d, dtype=dtype, device="cuda") for _ in range(2)]
    poss, counts, outs, graphs = [ints(*[0] * seqs) for _ in range(2)], [ints(*[0] * seqs) for _ in range(2)], [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        outs.append(torch.zeros_like(qs[i]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            cache.attention(qs[i], poss[i], counts=counts[i], rope_theta=10000.0, out=outs[i], workspace=ws[i])
    for turn in range(6):
        g = torch.Generator().manual_seed(turn)
        for i in range(2):
            qs[i].copy_(normal((seqs, t, hq, d), 10 * turn + i).to(dtype))
            c = torch.randint(0, t + 1, (seqs,), generator=g, dtype=torch.int32)
            counts[i].copy_(c)
            poss[i].copy_((torch.rand(seqs, generator=g) * (n - c)).int())
            outs[i].zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], cache.attention(qs[i], poss[i], counts=counts[i], rope_theta=10000.0)), (turn, i)
    assert cache.error() == 0

@pytest.mark.parametrize("hq,hk,d", [(8, 2, 64), (12, 2, 128)])
def test_a_prompt_is_dealt_out_by_the_keys_that_its_rows_see(hq, hk, d):
    # T key tiles hold the prompt; a row tile from position 0 on sees T / 2 of them on average, one of as many rows behind the
    # prompt 3 T / 2. With a unit's own cost of up to 16 tiles, equal runs take (64 + 16) / (192 + 16) = 0.39 of the time at T = 128;
    # where every row tile counts by all of its T places, some warp has a run without empty ones: half
    n = 8192
    cache = filled(hk, d, [2 * n], 2 * n, E4M3, 64, seed=6, spread=0.3)
    q = normal((1, n, hq, d), 7).cuda()
    out, first, second = torch.zeros_like(q), ints(0), ints(n)
    ahead = time_of(lambda: cache.attention(q, first, out=out))
    behind = time_of(lambda: cache.attention(q, second, out=out))
    assert ahead < 0.45 * behind, (ahead, behind)

def test_python_layer_refuses_bad_tensors():
    cache = T.Kv8Cache(2, 64, 100, n_seqs=2)
    x, pos = torch.zeros(2, 3, 2, 64, device="cuda"), ints(0, 0)
    for bad in (dict(k=x[:1]), dict(k=x.cpu()), dict(k=x.double()), dict(v=x.half()), dict(k=x[..., ::2]), dict(v=x[:, :2]),
                dict(pos=pos.long()), dict(pos=pos[:1]), dict(pos=pos.cpu()), dict(k=torch.zeros(2, 3, 3, 64, device="cuda"))):
        with pytest.raises((ValueError, T.TinferError)):
            cache.append(**{**dict(k=x, v=x, pos=pos), **bad})
    with pytest.raises(T.TinferError):  # rows that do not lie on 16 bytes
        cache.append(torch.zeros(2, 3, 2, 65, device="cuda")[..., 1:], x, pos)
    with pytest.raises(T.TinferError):
        cache.attention(torch.zeros(2, 3, 3, 64, device="cuda"), pos)
    with pytest.raises(ValueError):
        cache.attention(x, pos, lse=torch.zeros(2, 3, 2, device="cuda", dtype=torch.float64))
    with pytest.raises(T.TinferError):
        cache.attention(x, pos, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(T.TinferError):
        T.Kv8Cache(2, 96, 100)
