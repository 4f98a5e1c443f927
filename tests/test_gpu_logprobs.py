"""Token log probabilities, entropies and alternatives on the GPU against plain ones in 64 bits.

Tolerance. A term e^z of the sums is off by |z| 2^-23 (its argument's rounding) and 2^-22 (the exponential), so
log S0 by sum p |z| 2^-23 + 2^-22, and by its additions: a thread adds at most 2^18 / 8 / 256 * 2 = 256 terms, then 8 + 8
+ 3 partial sums, 275 * 2^-24 < 2^-15.8. sum p |z| = log S0 - H-like and below 2^4 here. S1 / S0 is off by twice
the same relative to sum p |z|. Results round once or twice more."""
import math

import pytest

torch = pytest.importorskip("torch")

import decode_persistent_megakernel_gb300 as T  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu
SUM = 2.0 ** -15.8 + 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    T.build()


def reference(x, targets, k):
    """float64 on the CPU; equal logits by the lower id."""
    x = x.double().cpu()
    lse = torch.logsumexp(x, dim=1)
    p = torch.exp(x - lse[:, None])
    z = x - x.amax(dim=1, keepdim=True)
    h = lse - torch.where(p > 0, p * x, 0.0).sum(1)
    mean = torch.where(p > 0, p * z.abs(), 0.0).sum(1)
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    logp = x.gather(1, targets.cpu().long()[:, None])[:, 0] - lse
    return logp, h, i[:, :k], v[:, :k] - lse[:, None], mean


def check(x, k, seed=0):
    rows, vocab = x.shape
    targets = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
    logp, h, ids, top = T.logprobs(x, targets, top_k=k)
    rl, rh, ri, rt, mean = reference(x, targets, max(k, 1))
    assert bool(((logp.cpu().double() - rl).abs() <= SUM + rl.abs() * 2.0 ** -22)[rl.isfinite()].all())
    assert torch.equal(logp.cpu().isinf(), rl.isinf())
    assert bool(((h.cpu().double() - rh).abs() <= SUM * (2 + 2 * mean) + rh.abs() * 2.0 ** -22).all())
    if k:
        assert torch.equal(ids.cpu().long(), ri)
        assert bool(((top.cpu().double() - rt).abs() <= SUM + rt.abs() * 2.0 ** -22).all())
    else:
        assert ids is None and top is None


@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 63, 257, 2048, 32000, 49152, 128256, 151936, 262144])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_sizes_and_types(vocab, dtype):
    rows = 3
    x = (3 * torch.randn((rows, vocab), generator=torch.Generator().manual_seed(vocab))).to(dtype).cuda()
    for k in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        check(x, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first,pad", [(0, 1), (1, 0), (3, 5), (7, 2), (5, 8)])
def test_rows_at_any_alignment(dtype, first, pad):
    for vocab in (5, 100, 4001, 50001):
        buf = torch.full((6 * (vocab + pad) + first + 64,), 1e30, dtype=dtype, device="cuda")  # beside the rows: huge
        x = buf[first:first + 6 * (vocab + pad)].view(6, vocab + pad)[:, :vocab]
        x.copy_(torch.randn((6, vocab), generator=torch.Generator().manual_seed(first)))
        check(x, min(20, vocab))


@pytest.mark.parametrize("rows", [1, 7, 300, 2000])
def test_many_rows(rows):
    x = (2 * torch.randn((rows, 5000), generator=torch.Generator().manual_seed(rows))).cuda()
    check(x, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [40, 3001, 128256])
def test_equal_logits_go_by_the_lower_id(dtype, vocab):
    k = 32
    check(torch.zeros((2, vocab), dtype=dtype, device="cuda"), k)                    # all equal
    x = torch.zeros((2, vocab), dtype=dtype, device="cuda")
    x[0, ::2] = -0.0                                                                 # zeros of both signs
    check(x, k)
    x = torch.arange(vocab, device="cuda").remainder(7).to(dtype)[None].repeat(2, 1)  # many ties at the top
    check(x, k)
    check((torch.arange(vocab, device="cuda") * (1.0 / 1024)).to(dtype)[None], k)     # rising
    check((torch.arange(vocab, device="cuda") * (-1.0 / 1024)).to(dtype)[None], k)    # falling
    x = torch.zeros((1, vocab), dtype=dtype, device="cuda")
    x[0, ::1024] = 1.0  # the large ones in the hands of few threads
    x[0, 1::1024] = 1.0
    check(x, k)


def test_masked_tokens():
    g = torch.Generator().manual_seed(3)
    for vocab, left in ((100, 3), (100, 1), (50000, 2), (50000, 40), (128256, 1000)):
        x = torch.randn((4, vocab), generator=g)
        keep = torch.randperm(vocab, generator=g)[:left]
        y = torch.full_like(x, -math.inf)
        y[:, keep] = x[:, keep]
        y = y.cuda()
        targets = keep[:1].repeat(4).int().cuda()
        k = 8
        logp, h, ids, top = T.logprobs(y, targets, top_k=k)
        rl, rh, ri, rt, _ = reference(y, targets, k)
        n = min(k, left)
        assert bool(((logp.cpu().double() - rl).abs() <= SUM + rl.abs() * 2.0 ** -22).all())
        assert bool(((h.cpu().double() - rh).abs() <= SUM * 20).all())
        assert torch.equal(ids.cpu()[:, :n].long(), ri[:, :n])
        assert bool((ids[:, n:] == -1).all()) and bool((top[:, n:] == -math.inf).all())
        hidden = torch.tensor([next(i for i in range(vocab) if i not in set(keep.tolist()))] * 4).int().cuda()
        assert bool((T.logprobs(y, hidden)[0] == -math.inf).all())


def test_rows_that_say_nothing():
    x = torch.randn((6, 3000), generator=torch.Generator().manual_seed(1))
    x[1] = -math.inf
    x[2, 77] = math.nan
    x[3, 2999] = math.inf
    x[4] = math.nan
    x[5, :] = -math.inf
    x[5, 1500] = math.nan
    targets = torch.tensor([0, 5, 5, 5, 5, 5], dtype=torch.int32, device="cuda")
    logp, h, ids, top = (t.cpu() for t in T.logprobs(x.cuda(), targets, top_k=4))
    assert logp[0].isfinite() and h[0].isfinite() and bool((ids[0] >= 0).all())
    assert logp[1] == -math.inf and h[1] == 0 and bool((ids[1] == -1).all()) and bool((top[1] == -math.inf).all())
    for r in (2, 3, 4, 5):
        assert logp[r].isnan() and h[r].isnan() and bool((ids[r] == -1).all()) and bool(top[r].isnan().all()), r


def test_targets_outside_the_vocabulary():
    x = torch.randn((4, 1000), generator=torch.Generator().manual_seed(1)).cuda()
    targets = torch.tensor([-1, 1000, -(2 ** 31), 999], dtype=torch.int32, device="cuda")
    logp, h, _, _ = T.logprobs(x, targets)
    assert logp[:3].isnan().all() and logp[3].isfinite() and h.isfinite().all()


def test_huge_and_tiny_logits():
    x = torch.randn((3, 4000), generator=torch.Generator().manual_seed(2))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2, 5] = 3e38
    targets = torch.tensor([3, 3, 5], dtype=torch.int32).cuda()
    logp, h, ids, top = T.logprobs(x.cuda(), targets, top_k=2)
    rl, rh, ri, rt, _ = reference(x, targets, 2)
    assert torch.equal(ids.cpu().long(), ri)
    assert bool(((logp.cpu().double() - rl).abs() <= SUM + rl.abs() * 2.0 ** -22).all())
    assert bool(((h.cpu().double() - rh).abs() <= SUM * 20).all())


def test_streams_and_graphs():
    x = torch.randn((5, 32000), generator=torch.Generator().manual_seed(2)).cuda()
    t = torch.arange(5, dtype=torch.int32, device="cuda")
    want = T.logprobs(x, t, top_k=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = T.logprobs(x, t, top_k=6)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = T.logprobs(buf, t, top_k=6)
    buf.copy_(x)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# From 229 rows on (152 multiprocessors) one CTA of 512 threads walks a whole row. At 2^18 logits a thread adds 512
# terms and 9 joins follow, 521 * 2^-24; its sums are rescaled by each of 2^18 / 512 / 16 = 32 turns at most, each time
# off by the exponential and two roundings, 32 * (2^-22 + 2^-23); the rest as above.
ROW_SUM = 521 * 2.0 ** -24 + 32 * (2.0 ** -22 + 2.0 ** -23) + 2.0 ** -18


def check_whole_rows(x, k, seed=0):
    rows, vocab = x.shape
    targets = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
    logp, h, ids, top = T.logprobs(x, targets, top_k=k)
    for a in range(0, rows, 128):  # (the reference on the GPU: elementary operations in 64 bits)
        y = x[a:a + 128].double()
        m = y.amax(dim=1, keepdim=True)
        e = torch.exp(y - m)
        norm = torch.log(e.sum(dim=1))
        p = e / e.sum(dim=1, keepdim=True)
        z = (m - y).clamp_max(1e30)
        mean = torch.where(p > 0, p * z, 0.0).sum(dim=1)
        want = (y - m).gather(1, targets[a:a + 128].long()[:, None])[:, 0] - norm
        assert bool(((logp[a:a + 128] - want).abs() <= ROW_SUM + want.abs() * 2.0 ** -22)[want.isfinite()].all())
        assert torch.equal(logp[a:a + 128].isinf(), want.isinf())
        assert bool(((h[a:a + 128] - norm - mean).abs() <= ROW_SUM * (2 + 2 * mean) + (norm + mean) * 2.0 ** -22).all())
        if k:
            v, i = torch.sort(y, dim=1, descending=True, stable=True)
            assert torch.equal(ids[a:a + 128].long(), i[:, :k])
            t = v[:, :k] - m - norm[:, None]
            assert bool(((top[a:a + 128] - t).abs() <= ROW_SUM + t.abs() * 2.0 ** -22).all())


@pytest.mark.parametrize("k", [0, 1, 20, 32])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,vocab,pad", [(230, 128256, 0), (600, 128256, 3), (256, 262144, 0), (150, 151936, 8), (100, 262144, 0)])
def test_many_rows_of_large_vocabularies(rows, vocab, pad, dtype, k):
    g = torch.Generator(device="cuda").manual_seed(rows + k)
    x = (2.5 * torch.randn((rows, vocab + pad), generator=g, device="cuda")).to(dtype)[:, :vocab]
    x[:, torch.randperm(vocab, generator=g, device="cuda")[:500]] = -math.inf
    check_whole_rows(x, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [128256, 262144])
def test_many_rows_with_ties_and_rising_logits(vocab, dtype):
    rows, k, i = 240, 32, torch.arange(vocab, device="cuda")
    x = torch.zeros((rows, vocab), dtype=dtype, device="cuda")
    x[1::6] = (i % 7).to(dtype)                 # thousands of equal largest logits: more than are listed
    x[2::6] = (i * (20.0 / vocab)).to(dtype)    # rising: every turn's maximum is a new one
    x[3::6] = (i * (-20.0 / vocab)).to(dtype)
    x[4::6, ::1024] = 1.0                       # the large ones in the hands of few threads
    x[5::6, 5:5 + 600] = 3.0                    # more equal ones side by side than are listed
    check_whole_rows(x, k)
    x[:, ::2] = -math.inf                       # and half of the tokens masked
    check_whole_rows(x, k)

def test_no_rows_give_empty_results():
    logp, h, ids, top = T.logprobs(torch.zeros((0, 500), device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), top_k=3)
    assert logp.shape == (0,) and h.shape == (0,) and ids.shape == (0, 3) and top.shape == (0, 3)
    for bad in (dict(logits=torch.zeros((0, 500), device="cuda"), top_k=33), dict(logits=torch.zeros((0, 500), device="cuda").double())):
        with pytest.raises((ValueError, T.TinferError)):
            T.logprobs(**bad)

@pytest.mark.parametrize("rows,vocab,dtype", [(1, 600, torch.bfloat16), (1, 2048, torch.bfloat16), (64, 2048, torch.float16),
                                              (500, 1000, torch.float32), (500, 2048, torch.bfloat16)])
def test_alternatives_of_a_small_vocabulary_take_no_pass_each(rows, vocab, dtype):
    # 32 alternatives by a floor and ranks, not by one maximum after another: far less than 32 times what one costs more
    x = (2.5 * torch.randn((rows, vocab), generator=torch.Generator().manual_seed(vocab))).to(dtype).cuda()
    check(x, 32)
    graphs, stream = [], torch.cuda.Stream()
    for k in (1, 32):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            for _ in range(20):
                T.logprobs(x, None, top_k=k)
    times = []
    for g in graphs:
        g.replay()
        runs = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            g.replay()
            b.record()
            b.synchronize()
            runs.append(a.elapsed_time(b))
        times.append(sorted(runs)[2])
    assert times[1] < 3 * times[0], times

def test_scores_of_the_decode_step():
    # the engine's logits of a step: its greedy token is the first alternative, its log probability the target's
    cfg = synth.config("tiny", max_ctx=8)
    eng = T.Engine(cfg, synth.make_model(cfg, seed=0), T.TINFER_MEGAKERNEL, kv=synth.make_kv(cfg, 0))
    eng.step(3, 0)
    logp, h, ids, top = T.logprobs(eng.logits[None], eng.argmax, top_k=1)
    torch.cuda.synchronize()
    assert int(ids) == int(eng.argmax) and float(top) == float(logp) and float(h) > 0
    rl, rh, _, _, _ = reference(eng.logits[None], eng.argmax, 1)
    assert abs(float(logp) - float(rl)) <= SUM + abs(float(rl)) * 2.0 ** -22
    eng.close()


def test_python_layer_refuses_bad_tensors():
    x = torch.zeros((2, 10), device="cuda")
    for bad in (dict(logits=x[0]), dict(logits=x.t()), dict(logits=x.double()), dict(targets=torch.zeros(2, device="cuda")),
                dict(targets=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(top_k=33)):
        with pytest.raises((ValueError, T.TinferError)):
            T.logprobs(**{**dict(logits=x), **bad})
