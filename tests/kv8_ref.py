"""Plain 64-bit implementations of the 8-bit KV cache operators, and the bounds of the kernels' roundings
(torch on the CPU; no code of the package)."""
import math

import torch

QMAX = {0: 448.0, 1: 127.0}  # TINFER_KV8_E4M3, TINFER_KV8_INT8


def nearest(x, fmt):
    """Nearest value of the format, ties to even, saturating; x float64."""
    if fmt == 1:
        return torch.round(x).clamp(-127, 127)
    _, e = torch.frexp(x)
    step = torch.exp2(((e - 1).clamp_min(-6) - 3).double())
    return (torch.round(x / step) * step).clamp(-448, 448)


def half_step(x, fmt):
    """Half the distance of neighbouring values of the format at x."""
    if fmt == 1:
        return torch.full_like(x, 0.5)
    _, e = torch.frexp(x)
    return 0.5 * torch.exp2(((e - 1).clamp_min(-6) - 3).double())


def decode(codes, fmt):
    c = codes.cpu()
    return (c.view(torch.float8_e4m3fn).float() if fmt == 0 else c.view(torch.int8)).double()


def rotate(x, first, theta):
    """x [t][h][d] float64 at positions first .. first + t - 1."""
    if not theta:
        return x
    t, h, d = x.shape
    f = torch.tensor([theta ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64)
    a = torch.outer(torch.arange(first, first + t, dtype=torch.float64), f)[:, None, :]
    c, s = torch.cos(a), torch.sin(a)
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1)


def store(x, codes, scales, pos, fmt, block):
    """x [t][h][d] (float32 values, rotated already) into codes [h][ctx][d] (float64 values in units of
    the scale) and scales [h][blocks] (float64 holding float32 values), as tinfer_op_kv8_append is defined: amax
    / QMAX and x / scale rounded to float32."""
    qmax, at, end = QMAX[fmt], pos, pos + x.shape[0]
    x = x.float()
    while at < end:
        b = at // block
        to = min(end, (b + 1) * block)
        rows = x[at - pos:to - pos].transpose(0, 1)
        for h in range(x.shape[1]):
            r = rows[h]
            amax = float(r.abs().max())
            held = float(scales[h, b]) if at > b * block else 0.0
            if not bool(torch.isfinite(r).all()) or math.isnan(held):
                scales[h, b] = math.nan
                codes[h, at:to] = 0
                continue
            if held > 0:
                s = held
                while amax > qmax * s:
                    s *= 2
                if s != held:
                    codes[h, b * block:at] = nearest(codes[h, b * block:at] * (held / s), fmt)
            else:
                s = max(float(torch.tensor(amax) / torch.tensor(qmax)), 2.0 ** -126) if amax > 0 else 0.0
            scales[h, b] = s
            codes[h, at:to] = nearest((r / torch.tensor(s, dtype=torch.float32)).double(), fmt) if s > 0 else 0
        at = to


def attend(q, k, v, pos):
    """q [t][hq][d], k and v [hk][n][d], float64; token i sees positions [0, pos + i]. Returns the outputs, the
    logarithms of the sums, the products' size sum |q||k| / sqrt(d) at most, and sum p |v|."""
    t, hq, d = q.shape
    g = hq // k.shape[0]
    n = k.shape[1]
    late = torch.arange(n)[None, :] > pos + torch.arange(t)[:, None]
    out, lse, size, mean = torch.empty_like(q), torch.empty((t, hq), dtype=torch.float64), torch.empty((t, hq), dtype=torch.float64), torch.empty_like(q)
    for h in range(hq):
        kk, vv = k[h // g], v[h // g]
        s = (q[:, h] @ kk.T / math.sqrt(d)).masked_fill(late, -math.inf)
        p = torch.softmax(s, dim=1)
        out[:, h], mean[:, h], lse[:, h] = p @ vv, p @ vv.abs(), torch.logsumexp(s, dim=1)
        size[:, h] = ((q[:, h].abs() @ kk.abs().T) / math.sqrt(d)).masked_fill(late, 0).amax(dim=1)
    return out, lse, size, mean


def attend_bounds(out, size, mean, d, n, dtype, top):
    """How far a kernel's outputs and log-sums may be from attend()'s. A score is off by at most
    (e_q + (d + 8) 2^-23) * size: the query's rounding (two fp16 parts: 2^-22, one: 2^-11), its rotation
    in fp32 (angle and products: below 2^-20), and a fp32 sum of d products that may truncate; its scaling
    by three fp32 factors. A weight e^score is off by that, by 2^-21 for the exponential and its argument
    (scores up to 2^6 in units of log 2 off by 2^-18 * size at most are within e_q), and by its rounding to
    fp16 parts (2^-22 or 2^-11). The weights enter twice (numerator and sum), the sum of n products
    truncates by (n + 64) 2^-23 at worst in sequence; rounding the result adds half a step. A weight far below
    the row's largest is held in fp16 steps of 2^-24 with the largest (times its V scale's power of two) near
    2^14, so it is off by up to 2^-25 of that whatever its size: 2^-39 of the largest weight, and n of them times
    the largest code by n 2^-38 top, `top` the largest V scale times the largest V code. It shows
    where one key has nearly all the weight and a code 0."""
    wide = dtype != torch.bfloat16
    e_score = (2.0 ** -19 if wide else 2.0 ** -11 + 2.0 ** -19) + (d + 8) * 2.0 ** -23
    e_weight = torch.expm1(e_score * size) + (2.0 ** -20 if wide else 2.0 ** -11 + 2.0 ** -20)
    e_sum = (min(n, 4096) + 64) * 2.0 ** -23
    far = (2 * e_weight[..., None] + e_sum) * mean
    # rounding to fp16: its numbers below 2^-14 are 2^-24 apart, so a result there is off by up to 2^-25
    # whatever its size (an output of 1.6e-11 is 0 in fp16); fp32 and bf16 reach down to 2^-126
    floor = 2.0 ** -25 if dtype == torch.float16 else 1e-30
    return far + out.abs() * torch.finfo(dtype).eps / 2 + floor + n * 2.0 ** -38 * top, e_score * size + e_sum + 2.0 ** -20
