"""The entry points around a step (head norms, mixture-of-experts layer, sampling) on the CPU: every argument that the
host can check is refused before the first CUDA call, so the stand-in addresses are never dereferenced."""
import pytest

import decode_persistent_megakernel_gb300 as T

A = 1 << 20  # aligned stand-in address
BAD, NO = T.TINFER_ERR_INVALID_ARG, T.TINFER_ERR_UNSUPPORTED
F32, F16, BF16 = T.TINFER_DTYPE_F32, T.TINFER_DTYPE_F16, T.TINFER_DTYPE_BF16


@pytest.fixture(scope="module", autouse=True)
def built():
    T.build()


def rows(data=A, dtype=BF16, ss=8192, ts=512, hs=64):
    return T.tinfer_rows(data, dtype, ss, ts, hs)


def norm(n_seqs=2, n_tokens=3, n_heads=4, n_kv_heads=2, head_dim=64, rotary_dim=64, q=None, k=None, q_gain=A, k_gain=A,
         eps=1e-6, theta=1e4, pos=A, counts=None, q_out=None, k_out=None, status=None):
    q, k, q_out, k_out = q or rows(), k or rows(), q_out or rows(2 * A), k_out or rows(3 * A)
    return T.tinfer_op_qk_norm_rope(n_seqs, n_tokens, n_heads, n_kv_heads, head_dim, rotary_dim, q, k, q_gain, k_gain, eps,
                                    theta, pos, counts, q_out, k_out, status)


@pytest.mark.parametrize("over,want", [
    (dict(n_seqs=0), BAD), (dict(n_tokens=0), BAD), (dict(n_heads=0), BAD), (dict(n_kv_heads=0), BAD),
    (dict(head_dim=0), BAD), (dict(pos=None), BAD), (dict(pos=A + 2), BAD), (dict(counts=A + 1), BAD),
    (dict(status=A + 2), BAD), (dict(q_gain=A + 2), BAD), (dict(k_gain=A + 1), BAD), (dict(eps=-1e-6), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(theta=0.5), BAD), (dict(theta=-1.0), BAD),
    (dict(theta=float("nan")), BAD), (dict(rotary_dim=-2), BAD), (dict(rotary_dim=80), BAD), (dict(rotary_dim=33), BAD),
    (dict(rotary_dim=24), NO), (dict(head_dim=72, rotary_dim=64), NO), (dict(head_dim=272), NO), (dict(n_heads=1025), NO),
    (dict(n_kv_heads=1025), NO), (dict(q=rows(None)), BAD), (dict(q=rows(A + 8)), BAD), (dict(k=rows(hs=68)), BAD),
    (dict(k=rows(ts=-512)), BAD), (dict(q=rows(dtype=3)), BAD), (dict(q=rows(dtype=F32)), BAD),
    (dict(q_out=rows(2 * A, dtype=F32)), BAD), (dict(q_out=rows(2 * A, hs=0)), BAD), (dict(k_out=rows(3 * A, ts=64)), BAD),
    (dict(q_out=rows(2 * A), k_out=rows(2 * A)), BAD),
    (dict(q_out=rows(2 * A, dtype=F16), k_out=rows(3 * A, dtype=F16)), NO),
])
def test_head_norms_refuse(over, want):
    assert norm(**over) == want
