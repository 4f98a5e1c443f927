"""The 8-bit KV cache and token-score entry points on the CPU: every argument that the host can check is refused
before the first CUDA call, so the stand-in addresses are never dereferenced."""
import ctypes

import pytest
import torch

import decode_persistent_megakernel_gb300 as T
import kv8_ref as R

A = 1 << 20  # aligned stand-in address
BAD, NO = T.TINFER_ERR_INVALID_ARG, T.TINFER_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    T.build()


def cache(**over):
    c = dict(format=T.TINFER_KV8_E4M3, n_seqs=2, n_kv_heads=2, head_dim=64, max_ctx=100, block=32, k_codes=A,
             v_codes=A, k_scales=A, v_scales=A)
    c.update(over)
    return T.tinfer_kv8(*(c[n] for n, _ in T.tinfer_kv8._fields_))


def rows(data=A, dtype=T.TINFER_DTYPE_BF16, ss=4096, ts=256, hs=64):
    return T.tinfer_rows(data, dtype, ss, ts, hs)


def every(c, n_tokens=3, pos=A, k=None, v=None, theta=0.0, n_heads=4, ws=A, ws_bytes=1 << 30, lse=None):
    k, v = k or rows(), v or rows()
    return (T.tinfer_op_kv8_append(c, k, v, n_tokens, pos, None, theta),
            T.tinfer_op_kv8_read(c, n_tokens, pos, None, k, v),
            T.tinfer_op_kv8_attention(c, n_heads, n_tokens, k, pos, None, theta, v, lse, ws, ws_bytes))


@pytest.mark.parametrize("over,want", [
    (dict(format=2), BAD), (dict(format=-1), BAD), (dict(n_seqs=0), BAD), (dict(n_kv_heads=0), BAD),
    (dict(max_ctx=0), BAD), (dict(block=8), BAD), (dict(block=48), BAD), (dict(block=256), BAD),
    (dict(k_codes=None), BAD), (dict(v_scales=None), BAD), (dict(k_codes=A + 8), BAD), (dict(v_codes=A + 4), BAD),
    (dict(k_scales=A + 2), BAD), (dict(head_dim=32), NO), (dict(head_dim=96), NO), (dict(head_dim=256), NO),
    (dict(n_seqs=1025), NO), (dict(max_ctx=(1 << 24) + 1), NO), (dict(n_kv_heads=1025), NO),
])
def test_bad_caches_are_refused(over, want):
    assert every(cache(**over)) == (want,) * 3
    assert T.tinfer_kv8_attention_workspace(cache(**over), 4, 1) == 0


@pytest.mark.parametrize("over", [
    dict(n_tokens=0), dict(n_tokens=-1), dict(n_tokens=101), dict(pos=None), dict(k=rows(data=None)),
    dict(k=rows(data=A + 8)), dict(v=rows(data=A + 2)), dict(k=rows(dtype=3)), dict(k=rows(ss=-4096)),
    dict(k=rows(ts=260)), dict(k=rows(hs=68)), dict(v=rows(dtype=T.TINFER_DTYPE_F32)),
    dict(k=rows(dtype=T.TINFER_DTYPE_F32, ts=258), v=rows(dtype=T.TINFER_DTYPE_F32)),
])
def test_bad_rows_are_refused(over):
    assert every(cache(), **over) == (BAD,) * 3


def test_written_rows_must_not_overlap():
    for r in (rows(hs=56), rows(ts=0), rows(ss=8)):
        assert T.tinfer_op_kv8_read(cache(), 3, A, None, rows(), r) == BAD
        assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), A, None, 0.0, r, None, A, 1 << 30) == BAD


@pytest.mark.parametrize("ss,ts,hs", [(4096, 64, 64), (512, 256, 128), (128, 4096, 128), (256, 64, 256)])
def test_written_rows_that_share_memory_are_refused(ss, ts, hs):
    r = rows(ss=ss, ts=ts, hs=hs)  # each stride holds a row, but two rows of [2][3][4] (or [2][3][2]) meet
    assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), A, None, 0.0, r, None, A, 1 << 30) == BAD
    assert T.tinfer_op_kv8_read(cache(n_kv_heads=4), 3, A, None, rows(), r) == BAD


def test_results_over_the_queries_want_their_strides():
    assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), A, None, 0.0, rows(ts=512), None, A, 1 << 30) == BAD


@pytest.mark.parametrize("at", ["pos", "counts", "status"])
def test_words_off_their_boundary_are_refused(at):
    a = dict(pos=A, counts=A, status=A)
    a[at] = A + 2
    assert T.tinfer_op_kv8_append(cache(), rows(), rows(), 3, a["pos"], a["counts"], 0.0, a["status"]) == BAD
    assert T.tinfer_op_kv8_read(cache(), 3, a["pos"], a["counts"], rows(), rows(), a["status"]) == BAD
    assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), a["pos"], a["counts"], 0.0, rows(2 * A), None, A, 1 << 30,
                                     a["status"]) == BAD


def test_bad_angles_heads_and_workspaces_are_refused():
    for theta in (-1.0, 0.5, float("nan"), float("inf")):
        assert T.tinfer_op_kv8_append(cache(), rows(), rows(), 3, A, None, theta) == BAD
        assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), A, None, theta, rows(), None, A, 1 << 30) == BAD
    for n_heads in (0, 3, -2):
        assert T.tinfer_op_kv8_attention(cache(), n_heads, 3, rows(), A, None, 0.0, rows(), None, A, 1 << 30) == BAD
        assert T.tinfer_kv8_attention_workspace(cache(), n_heads, 3) == 0
    need = T.tinfer_kv8_attention_workspace(cache(), 4, 3)
    assert need > 0
    for ws, n in ((None, need), (A + 8, need), (A, need - 1)):
        assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), A, None, 0.0, rows(), None, ws, n) == BAD
    assert T.tinfer_op_kv8_attention(cache(), 4, 3, rows(), A, None, 0.0, rows(), A + 2, A, need) == BAD
    big = cache(n_seqs=1024, n_kv_heads=1024, max_ctx=1 << 24)
    assert T.tinfer_op_kv8_attention(big, 1024, 1, rows(), A, None, 0.0, rows(2 * A, ss=65536), None, A, 1 << 40) == NO


def test_no_workspace_for_what_every_attention_refuses():
    ws = T.tinfer_kv8_attention_workspace
    assert ws(cache(), 4, 100) > 0 and ws(cache(), 4, 101) == 0               # more tokens than the cache holds
    big = dict(n_seqs=128, n_kv_heads=1, max_ctx=1 << 24)                    # 2^31 rows, and one sequence less
    assert ws(cache(**big), 1, 1) == 0 and ws(cache(**{**big, "n_seqs": 127}), 1, 1) > 0
    assert ws(cache(n_kv_heads=1, max_ctx=1 << 24, n_seqs=1), 65, 1 << 24) == 0  # more than 2^30 query rows of a KV head
    for c, heads, tokens in ((cache(**big), 1, 1), (cache(n_kv_heads=1, max_ctx=1 << 24, n_seqs=1), 65, 1 << 24)):
        for dtype in (T.TINFER_DTYPE_F32, T.TINFER_DTYPE_BF16):
            r = rows(dtype=dtype, ss=1 << 40, ts=1 << 14, hs=64)
            assert T.tinfer_op_kv8_attention(c, heads, tokens, r, A, None, 0.0, r, None, A, 1 << 30) in (NO, BAD)


def test_a_cache_that_every_attention_refuses_is_not_made():
    with pytest.raises(T.TinferError):  # refused before 275 GB are asked for
        T.Kv8Cache(1, 64, 1 << 24, n_seqs=128)
    with pytest.raises(T.TinferError):
        T.Kv8Cache(1, 64, 100, fmt=5)

def test_keys_and_values_written_to_one_place_are_refused():
    r = rows(ss=1024)
    assert T.tinfer_op_kv8_read(cache(), 3, A, None, r, r) == BAD
    k = rows(2 * A)
    for same in (dict(v_codes=A, k_scales=2 * A), dict(v_scales=2 * A, k_scales=2 * A, k_codes=3 * A)):
        assert T.tinfer_op_kv8_append(cache(**same), k, k, 3, A, None, 0.0) == BAD

@pytest.mark.parametrize("over,want", [
    (dict(rows=0), BAD), (dict(vocab=0), BAD), (dict(dtype=7), BAD), (dict(logits=None), BAD), (dict(logits=A + 2), BAD),
    (dict(row_stride=99), BAD), (dict(top_k=-1), BAD), (dict(top_k=33), BAD), (dict(targets=None), BAD),
    (dict(top_ids=None), BAD), (dict(top_logp=None), BAD), (dict(top_k=0), BAD), (dict(entropy=A + 2), BAD),
    (dict(targets=A + 1), BAD), (dict(vocab=(1 << 18) + 1, row_stride=1 << 19), NO),
])
def test_bad_score_arguments_are_refused(over, want):
    a = dict(rows=2, vocab=100, dtype=T.TINFER_DTYPE_F32, logits=A, row_stride=100, targets=A, top_k=3, logp=A,
             entropy=A, top_ids=A, top_logp=A)
    a.update(over)
    assert T.tinfer_op_logprobs(*a.values()) == want


def test_nothing_asked_for_is_refused():
    assert T.tinfer_op_logprobs(2, 100, 0, A, 100, None, 0, None, None, None, None) == BAD


def test_null_structures_are_refused():
    lib, r = T.lib(), rows()
    assert lib.tinfer_op_kv8_append(None, r, r, 1, A, None, 0.0, None, None) == BAD
    assert lib.tinfer_op_kv8_append(cache(), None, r, 1, A, None, 0.0, None, None) == BAD
    assert lib.tinfer_op_kv8_read(cache(), 1, A, None, r, None, None, None) == BAD
    assert lib.tinfer_kv8_attention_workspace(None, 4, 1) == 0


def test_structures_match_the_header():
    assert ctypes.sizeof(T.tinfer_kv8) == 6 * 4 + 4 * 8
    assert ctypes.sizeof(T.tinfer_rows) == 8 + 8 + 3 * 8


def test_python_layer_refuses_host_tensors():
    with pytest.raises(ValueError):
        T.Kv8Cache(2, 64, 100, device="cpu")
    with pytest.raises(ValueError):
        T.logprobs(torch.zeros(2, 10))


def test_reference_rounding():
    # the reference's e4m3 rounding against torch's on every tie and neighbour of the positive codes
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (v[1:] + v[:-1]) / 2
    for x in (v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)):
        assert torch.equal(R.nearest(x, 0), x.float().to(torch.float8_e4m3fn).double())
    assert R.nearest(torch.tensor([1e6, -1e6], dtype=torch.float64), 0).tolist() == [448.0, -448.0]
