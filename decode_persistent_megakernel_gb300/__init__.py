"""Python binding of libtinfer.so, the GB300 batch-1 decode engine (include/tinfer.h).

The functions below carry the C names and only marshal arguments: every step of the decode path
runs in the library's CUDA kernels. PyTorch is used for device memory and streams. There is no
fallback: if the library is missing or the GPU is absent, calls raise.
"""
from __future__ import annotations

import ctypes
import os

from .build import build  # noqa: F401  (bound here once: a later import of the submodule leaves the name alone)

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtinfer.so")

TINFER_OK, TINFER_ERR_INVALID_ARG, TINFER_ERR_UNSUPPORTED, TINFER_ERR_CUDA, TINFER_ERR_OOM, \
    TINFER_ERR_NONFINITE, TINFER_ERR_TIMEOUT = range(7)
TINFER_BF16, TINFER_INT4 = 0, 1
TINFER_SCALE_FP16, TINFER_SCALE_BF16 = 0, 1
TINFER_MEGAKERNEL, TINFER_GRAPH = 0, 1
TINFER_Q_GRID, TINFER_Q_SMEM, TINFER_Q_RING_STAGES, TINFER_Q_SLOT_BYTES, TINFER_Q_KERNELS_PER_STEP, \
    TINFER_Q_TRACE_BYTES, TINFER_Q_BLOCK_THREADS = range(7)
TINFER_EPI_STORE, TINFER_EPI_RESIDUAL, TINFER_EPI_SWIGLU, TINFER_EPI_ARGMAX = range(4)
TINFER_S_INFLIGHT, TINFER_S_INFLIGHT_LM, TINFER_S_L2_LOOKAHEAD, TINFER_S_L2_PACE, TINFER_S_SYNC, TINFER_S_ATTN_CHUNKS = range(6)
TINFER_SYNC_STAMPS, TINFER_SYNC_GRID_BARRIER = 0, 1
TINFER_NOALLOC_SCRATCH_BYTES = 1 << 20
TINFER_KV8_E4M3, TINFER_KV8_INT8 = 0, 1
TINFER_KV8_KEEP_STATUS, TINFER_KV8_DEBUG_WITHHOLD = 0x100, 0x200
TINFER_DTYPE_F32, TINFER_DTYPE_F16, TINFER_DTYPE_BF16 = range(3)
TRACE_FIELDS = 10  # stamps per CTA and phase of the timeline (tinfer_set_trace)

EXPORTS = [
    "tinfer_status_string", "tinfer_check_config", "tinfer_packed_layer_bytes", "tinfer_pack_layer",
    "tinfer_unpack_layer", "tinfer_create", "tinfer_decode_step", "tinfer_decode_step_dev",
    "tinfer_generate", "tinfer_generate_dev", "tinfer_get_error", "tinfer_query", "tinfer_set_trace", "tinfer_set_timeout_ns",
    "tinfer_debug_withhold_results", "tinfer_set_schedule", "tinfer_get_schedule", "tinfer_destroy",
    "tinfer_packed_row_bytes", "tinfer_pack_matrix", "tinfer_op_gemv", "tinfer_op_attention",
    "tinfer_op_attention_noalloc", "tinfer_op_gemv_batch", "tinfer_moe_packed_bytes", "tinfer_pack_moe", "tinfer_op_moe",
    "tinfer_op_gemm_bf16", "tinfer_op_kv8_append", "tinfer_op_kv8_read", "tinfer_kv8_attention_workspace",
    "tinfer_op_kv8_attention", "tinfer_op_logprobs",
]


class TinferError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: tinfer status {status} ({status_string(status)})")


class tinfer_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "n_layers", "hidden", "n_heads", "n_kv_heads", "head_dim", "ffn", "vocab", "max_ctx")] + [
        ("rope_theta", ctypes.c_double), ("rms_eps", ctypes.c_double)] + [
        (n, ctypes.c_int) for n in ("weight_format", "group_size", "scale_dtype", "tied_embeddings",
                                    "qkv_bias", "exec_mode", "ffn_split")]


class tinfer_layer_src(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "wq", "wk", "wv", "wo", "wg", "wu", "wd", "sq", "sk", "sv", "so", "sg", "su", "sd",
        "bq", "bk", "bv", "g1", "g2")]


class tinfer_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("final_norm", ctypes.c_void_p), ("layer_blobs", ctypes.POINTER(ctypes.c_void_p))]


class tinfer_kv8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("format", "n_seqs", "n_kv_heads", "head_dim", "max_ctx", "block")] + [
        (n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")]


class tinfer_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int)] + [
        (n, ctypes.c_longlong) for n in ("seq_stride", "token_stride", "head_stride")]


_lib = None


def lib():
    """The loaded library. Raises if it has not been built: there is no other implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run decode_persistent_megakernel_gb300.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, D, Z, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_size_t, ctypes.c_longlong
        cfgp = ctypes.POINTER(tinfer_config)
        kvp, rowp = ctypes.POINTER(tinfer_kv8), ctypes.POINTER(tinfer_rows)
        sig = {
            "tinfer_status_string": ([I], ctypes.c_char_p),
            "tinfer_check_config": ([cfgp], I),
            "tinfer_packed_layer_bytes": ([cfgp], Z),
            "tinfer_pack_layer": ([cfgp, ctypes.POINTER(tinfer_layer_src), P, P], I),
            "tinfer_unpack_layer": ([cfgp, P, ctypes.POINTER(tinfer_layer_src), P], I),
            "tinfer_create": ([cfgp, ctypes.POINTER(tinfer_weights), P, P, ctypes.POINTER(P)], I),
            "tinfer_decode_step": ([P, ctypes.c_int32, ctypes.c_int32, P, P, P], I),
            "tinfer_decode_step_dev": ([P, P, ctypes.c_int32, P, P, P], I),
            "tinfer_generate": ([P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P], I),
            "tinfer_generate_dev": ([P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P], I),
            "tinfer_get_error": ([P], I),
            "tinfer_query": ([P, I], LL),
            "tinfer_set_trace": ([P, P], I),
            "tinfer_set_timeout_ns": ([P, LL], I),
            "tinfer_debug_withhold_results": ([P, I, I], I),
            "tinfer_set_schedule": ([P, I, LL], I),
            "tinfer_get_schedule": ([P, I], LL),
            "tinfer_destroy": ([P], None),
            "tinfer_packed_row_bytes": ([I, I, I], Z),
            "tinfer_pack_matrix": ([I, I, I, I, I, P, P, P, P], I),
            "tinfer_op_gemv": ([I, I, I, I, I, P, P, P, D, P, I, P, P, P], I),
            "tinfer_op_attention": ([I, I, I, I, D, I, I, P, P, P, P, P, P, P, P], I),
            "tinfer_op_attention_noalloc": ([I, I, I, I, D, I, I, P, P, P, P, P], I),
            "tinfer_op_gemv_batch": ([I, I, I, I, I, I, P, P, P, I, P, P], I),
            "tinfer_moe_packed_bytes": ([I, I, I, I, I, I], Z),
            "tinfer_pack_moe": ([I, I, I, I, I, I, P, P, P, P, P, P, P, P, P], I),
            "tinfer_op_moe": ([I, I, I, I, I, I, I, P, P, P, P, P, P, P, I, P, P], I),
            "tinfer_op_gemm_bf16": ([I, I, I, P, P, P, P], I),
            "tinfer_op_kv8_append": ([kvp, rowp, rowp, I, P, P, D, P, P], I),
            "tinfer_op_kv8_read": ([kvp, I, P, P, rowp, rowp, P, P], I),
            "tinfer_kv8_attention_workspace": ([kvp, I, I], Z),
            "tinfer_op_kv8_attention": ([kvp, I, I, rowp, P, P, D, rowp, P, P, Z, P, P], I),
            "tinfer_op_logprobs": ([I, I, I, P, LL, P, I, P, P, P, P, P], I),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().tinfer_status_string(int(s)).decode()


def _check(rc: int, what: str) -> int:
    if rc != TINFER_OK:
        raise TinferError(rc, what)
    return rc


def _ptr(t) -> int | None:
    """Device address of a torch tensor (or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


# ------------------------------------------------------------------ C entry points, same names

def tinfer_check_config(cfg: tinfer_config) -> int:
    return lib().tinfer_check_config(ctypes.byref(cfg))


def tinfer_packed_layer_bytes(cfg: tinfer_config) -> int:
    return lib().tinfer_packed_layer_bytes(ctypes.byref(cfg))


def tinfer_pack_layer(cfg, src: tinfer_layer_src, packed, stream=None) -> int:
    return lib().tinfer_pack_layer(ctypes.byref(cfg), ctypes.byref(src), _ptr(packed), _stream(stream))


def tinfer_unpack_layer(cfg, packed, dst: tinfer_layer_src, stream=None) -> int:
    return lib().tinfer_unpack_layer(ctypes.byref(cfg), _ptr(packed), ctypes.byref(dst), _stream(stream))


def tinfer_create(cfg, weights: tinfer_weights, k_cache, v_cache):
    out = ctypes.c_void_p()
    rc = lib().tinfer_create(ctypes.byref(cfg), ctypes.byref(weights), _ptr(k_cache), _ptr(v_cache),
                             ctypes.byref(out))
    return rc, out


def tinfer_decode_step(ctx, token: int, pos: int, stream=None, logits=None, argmax=None) -> int:
    return lib().tinfer_decode_step(ctx, int(token), int(pos), _stream(stream), _ptr(logits), _ptr(argmax))


def tinfer_decode_step_dev(ctx, token_dev, pos: int, stream=None, logits=None, argmax=None) -> int:
    return lib().tinfer_decode_step_dev(ctx, _ptr(token_dev), int(pos), _stream(stream), _ptr(logits),
                                        _ptr(argmax))


def tinfer_generate(ctx, first_token: int, pos0: int, n_steps: int, stream, tokens_host) -> int:
    """tokens_host: a ctypes int32 array or a writable numpy int32 array of length >= n_steps."""
    if hasattr(tokens_host, "ctypes"):
        ptr = tokens_host.ctypes.data
    else:
        ptr = ctypes.addressof(tokens_host)
    return lib().tinfer_generate(ctx, int(first_token), int(pos0), int(n_steps), _stream(stream), ptr)


def tinfer_generate_dev(ctx, first_token: int, pos0: int, n_steps: int, eos_token: int, stream, tokens_dev,
                        count_dev=None) -> int:
    return lib().tinfer_generate_dev(ctx, int(first_token), int(pos0), int(n_steps), int(eos_token),
                                     _stream(stream), _ptr(tokens_dev), _ptr(count_dev))


def tinfer_get_error(ctx) -> int:
    return lib().tinfer_get_error(ctx)


def tinfer_query(ctx, what: int) -> int:
    return lib().tinfer_query(ctx, what)


def tinfer_set_trace(ctx, trace_dev) -> int:
    return lib().tinfer_set_trace(ctx, _ptr(trace_dev))


def tinfer_set_timeout_ns(ctx, ns: int) -> int:
    return lib().tinfer_set_timeout_ns(ctx, int(ns))


def tinfer_debug_withhold_results(ctx, cta: int, phase: int) -> int:
    return lib().tinfer_debug_withhold_results(ctx, int(cta), int(phase))


def tinfer_set_schedule(ctx, knob: int, value: int) -> int:
    return lib().tinfer_set_schedule(ctx, int(knob), int(value))


def tinfer_get_schedule(ctx, knob: int) -> int:
    return lib().tinfer_get_schedule(ctx, int(knob))


def tinfer_destroy(ctx) -> None:
    lib().tinfer_destroy(ctx)


def tinfer_packed_row_bytes(fmt: int, cols: int, group: int) -> int:
    return lib().tinfer_packed_row_bytes(fmt, cols, group)


def tinfer_pack_matrix(fmt, group, scale_dtype, rows, cols, w, scales, packed, stream=None) -> int:
    return lib().tinfer_pack_matrix(fmt, group, scale_dtype, rows, cols, _ptr(w), _ptr(scales),
                                    _ptr(packed), _stream(stream))


def tinfer_op_gemv(fmt, group, scale_dtype, rows, cols, packed, x, gain, eps, bias, epilogue, y,
                   argmax, stream=None) -> int:
    return lib().tinfer_op_gemv(fmt, group, scale_dtype, rows, cols, _ptr(packed), _ptr(x), _ptr(gain),
                                float(eps), _ptr(bias), epilogue, _ptr(y), _ptr(argmax), _stream(stream))


def tinfer_op_attention(nq, nkv, d, max_ctx, theta, pos, n_chunks, qkv, k_layer, v_layer, out,
                        part_m=None, part_l=None, part_o=None, stream=None) -> int:
    return lib().tinfer_op_attention(nq, nkv, d, max_ctx, float(theta), pos, n_chunks, _ptr(qkv),
                                     _ptr(k_layer), _ptr(v_layer), _ptr(out), _ptr(part_m),
                                     _ptr(part_l), _ptr(part_o), _stream(stream))


def tinfer_op_attention_noalloc(nq, nkv, d, max_ctx, theta, pos, n_chunks, qkv, k_layer, v_layer,
                                out, stream=None) -> int:
    return lib().tinfer_op_attention_noalloc(nq, nkv, d, max_ctx, float(theta), pos, n_chunks,
                                             _ptr(qkv), _ptr(k_layer), _ptr(v_layer), _ptr(out),
                                             _stream(stream))


def tinfer_op_gemv_batch(fmt, group, scale_dtype, rows, cols, m, packed, x, bias, epilogue, y, stream=None) -> int:
    return lib().tinfer_op_gemv_batch(fmt, group, scale_dtype, rows, cols, m, _ptr(packed), _ptr(x), _ptr(bias),
                                      epilogue, _ptr(y), _stream(stream))


def tinfer_moe_packed_bytes(fmt, group, n_experts, hidden, ffn_e, which) -> int:
    return lib().tinfer_moe_packed_bytes(fmt, group, n_experts, hidden, ffn_e, which)


def tinfer_pack_moe(fmt, group, scale_dtype, n_experts, hidden, ffn_e, wg, sg, wu, su, wd, sd, gu_packed,
                    down_packed, stream=None) -> int:
    return lib().tinfer_pack_moe(fmt, group, scale_dtype, n_experts, hidden, ffn_e, _ptr(wg), _ptr(sg), _ptr(wu),
                                 _ptr(su), _ptr(wd), _ptr(sd), _ptr(gu_packed), _ptr(down_packed),
                                 _stream(stream))


def tinfer_op_moe(fmt, group, scale_dtype, n_experts, top_k, hidden, ffn_e, gu_packed, down_packed, ids, weights,
                  x, h, y, accumulate=0, status=None, stream=None) -> int:
    return lib().tinfer_op_moe(fmt, group, scale_dtype, n_experts, top_k, hidden, ffn_e, _ptr(gu_packed),
                               _ptr(down_packed), _ptr(ids), _ptr(weights), _ptr(x), _ptr(h), _ptr(y),
                               int(accumulate), _ptr(status), _stream(stream))


# ------------------------------------------------------------------ marshalling helpers

def tinfer_op_gemm_bf16(m, n, k, x, w, y, stream=None) -> int:
    return lib().tinfer_op_gemm_bf16(m, n, k, _ptr(x), _ptr(w), _ptr(y), _stream(stream))


def tinfer_op_kv8_append(cache: tinfer_kv8, k: tinfer_rows, v: tinfer_rows, n_tokens, pos, counts=None,
                         rope_theta=0.0, status=None, stream=None) -> int:
    return lib().tinfer_op_kv8_append(cache, k, v, n_tokens, _ptr(pos), _ptr(counts), rope_theta, _ptr(status),
                                      _stream(stream))


def tinfer_op_kv8_read(cache: tinfer_kv8, n_tokens, pos, counts, k: tinfer_rows, v: tinfer_rows, status=None,
                       stream=None) -> int:
    return lib().tinfer_op_kv8_read(cache, n_tokens, _ptr(pos), _ptr(counts), k, v, _ptr(status), _stream(stream))


def tinfer_kv8_attention_workspace(cache: tinfer_kv8, n_heads, n_tokens) -> int:
    return lib().tinfer_kv8_attention_workspace(cache, n_heads, n_tokens)


def tinfer_op_kv8_attention(cache: tinfer_kv8, n_heads, n_tokens, q: tinfer_rows, pos, counts, rope_theta,
                            out: tinfer_rows, lse, workspace, workspace_bytes, status=None, stream=None) -> int:
    return lib().tinfer_op_kv8_attention(cache, n_heads, n_tokens, q, _ptr(pos), _ptr(counts), rope_theta, out,
                                         _ptr(lse), _ptr(workspace), workspace_bytes, _ptr(status), _stream(stream))


def tinfer_op_logprobs(rows, vocab, dtype, logits, row_stride, targets, top_k, logp, entropy, top_ids, top_logp,
                       stream=None) -> int:
    return lib().tinfer_op_logprobs(rows, vocab, dtype, _ptr(logits), row_stride, _ptr(targets), top_k, _ptr(logp),
                                    _ptr(entropy), _ptr(top_ids), _ptr(top_logp), _stream(stream))


def make_config(c: dict, exec_mode: int = TINFER_MEGAKERNEL) -> tinfer_config:
    """tinfer_config from a workload description (synth.CONFIGS entries or the same keys)."""
    cfg = tinfer_config()
    for f in ("n_layers", "hidden", "n_heads", "n_kv_heads", "head_dim", "ffn", "vocab", "max_ctx"):
        setattr(cfg, f, int(c[f]))
    cfg.rope_theta = float(c["rope_theta"])
    cfg.rms_eps = float(c["rms_eps"])
    cfg.weight_format = TINFER_INT4 if c["weight_format"] == "int4" else TINFER_BF16
    cfg.group_size = int(c.get("group_size") or 0)
    cfg.scale_dtype = TINFER_SCALE_BF16 if c.get("scale_dtype") == "bf16" else TINFER_SCALE_FP16
    cfg.tied_embeddings = 1 if c.get("tied") else 0
    cfg.qkv_bias = 1 if c.get("qkv_bias") else 0
    cfg.exec_mode = int(exec_mode)
    cfg.ffn_split = 1 if c.get("ffn_split") else 0
    return cfg


class Engine:
    """Owns the device copies of a canonical model (torch tensors), the packed layers, the KV cache
    and one tinfer context. The model dict is synth.make_model's layout (numpy arrays)."""

    def __init__(self, c: dict, weights: dict, exec_mode: int = TINFER_MEGAKERNEL, device: str = "cuda",
                 kv=None):
        import numpy as np
        import torch
        self.c = c
        self.cfg = make_config(c, exec_mode)
        _check(tinfer_check_config(self.cfg), "tinfer_check_config")
        dev = torch.device(device)
        self.device = dev

        def up(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a)
            t = torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a)
            return t.to(dev)

        self.embed = up(weights["embed"])
        self.lm_head = self.embed if weights["lm_head"] is weights["embed"] else up(weights["lm_head"])
        self.final_norm = up(weights["final_norm"])
        nbytes = tinfer_packed_layer_bytes(self.cfg)
        if nbytes == 0:
            raise TinferError(TINFER_ERR_UNSUPPORTED, "tinfer_packed_layer_bytes")
        self.blobs = []
        int4 = c["weight_format"] == "int4"
        for L in weights["layers"]:
            src = tinfer_layer_src()
            keep = {}
            for name in ("wq", "wk", "wv", "wo", "wg", "wu", "wd"):
                keep[name] = up(L[name])
                setattr(src, name, _ptr(keep[name]))
                if int4:
                    sname = "s" + name[1]
                    keep[sname] = up(L[sname])
                    setattr(src, sname, _ptr(keep[sname]))
            if c.get("qkv_bias"):
                for b in ("bq", "bk", "bv"):
                    keep[b] = up(L[b])
                    setattr(src, b, _ptr(keep[b]))
            for g in ("g1", "g2"):
                keep[g] = up(L[g])
                setattr(src, g, _ptr(keep[g]))
            blob = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            _check(tinfer_pack_layer(self.cfg, src, blob, torch.cuda.current_stream(dev)), "tinfer_pack_layer")
            self.blobs.append(blob)
            torch.cuda.current_stream(dev).synchronize()  # canonical copies can go
        shape = (c["n_layers"], c["n_kv_heads"], c["max_ctx"], c["head_dim"])
        if kv is not None:
            self.k = up(kv[0]).view(shape)
            self.v = up(kv[1]).view(shape)
        else:
            self.k = torch.zeros(shape, dtype=torch.int16, device=dev)
            self.v = torch.zeros(shape, dtype=torch.int16, device=dev)
        arr = (ctypes.c_void_p * len(self.blobs))(*[b.data_ptr() for b in self.blobs])
        self._blob_arr = arr
        w = tinfer_weights()
        w.embed, w.lm_head, w.final_norm = _ptr(self.embed), _ptr(self.lm_head), _ptr(self.final_norm)
        w.layer_blobs = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
        self._w = w
        rc, ctx = tinfer_create(self.cfg, w, self.k, self.v)
        _check(rc, "tinfer_create")
        self.ctx = ctx
        self.logits = torch.empty(c["vocab"], dtype=torch.float32, device=dev)
        self.argmax = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, token: int, pos: int, stream=None, logits=True):
        rc = tinfer_decode_step(self.ctx, token, pos, stream, self.logits if logits else None, self.argmax)
        _check(rc, "tinfer_decode_step")

    def step_dev(self, token_dev, pos: int, stream=None, logits=True, argmax=None):
        rc = tinfer_decode_step_dev(self.ctx, token_dev, pos, stream, self.logits if logits else None,
                                    self.argmax if argmax is None else argmax)
        _check(rc, "tinfer_decode_step_dev")

    def trace_step(self, token: int, pos: int):
        """Runs one traced megakernel step; returns int64 stamps [grid][phases][fields] (ns,
        relative to the earliest stamp; 0 stays 0 where nothing was recorded)."""
        import numpy as np
        import torch
        nbytes = self.query(TINFER_Q_TRACE_BYTES)
        buf = torch.zeros(nbytes // 8, dtype=torch.int64, device=self.device)
        _check(tinfer_set_trace(self.ctx, buf), "tinfer_set_trace")
        self.step(token, pos)
        torch.cuda.synchronize()
        _check(tinfer_set_trace(self.ctx, None), "tinfer_set_trace")
        t = buf.cpu().numpy().reshape(self.query(TINFER_Q_GRID), -1, TRACE_FIELDS)
        return np.where(t > 0, t - t[t > 0].min(), 0)

    def error(self) -> int:
        return tinfer_get_error(self.ctx)

    def query(self, what: int) -> int:
        return tinfer_query(self.ctx, what)

    def close(self):
        if getattr(self, "ctx", None):
            tinfer_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------ the 8-bit cache and token scores on tensors

_DTYPES: dict = {}  # torch dtype -> TINFER_DTYPE_*


def _dtype(t) -> int:
    """TINFER_DTYPE_* of a tensor (ValueError for the others)."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: TINFER_DTYPE_F32, torch.float16: TINFER_DTYPE_F16, torch.bfloat16: TINFER_DTYPE_BF16})
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"float32, float16 or bfloat16 is wanted, got {t.dtype}")
    return d


def _call(what, fn, args, device, stream) -> None:
    """Calls fn(*args, stream) with `device` current, on `stream` or torch's current one; raises on an error status.
    The raw getters are what torch.cuda's own wrappers call: a step's small calls are a few microseconds on the GPU."""
    import torch
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != TINFER_OK:
        raise TinferError(rc, what)


def _making(stream, device):
    """Context in which new results of a call on `stream` are made: their memory and first values belong to that stream."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _on(what: str, t, device, dtype=None, shape=None):
    """Checks a tensor argument: its device, and its dtype and shape where given."""
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what}: {dtype} is wanted, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} is wanted, got {tuple(t.shape)}")


class Kv8Cache:
    """An 8-bit KV cache of n_seqs sequences on one device, and the operators on it (tinfer_op_kv8_*). Rows are
    tensors [n_seqs, n_tokens, heads, head_dim] with contiguous rows, of any strides that keep each row on 16
    bytes. pos and counts are int32 tensors [n_seqs] on the device; pos[s] is where the first of the call's
    tokens of sequence s stands. Work runs on `stream`, or on torch's current stream of the device.

    buffers: (k_codes, v_codes, k_scales, v_scales) to use instead of new ones: uint8
    [n_seqs, n_kv_heads, max_ctx, head_dim] and float32 [n_seqs, n_kv_heads, ceil(max_ctx / block)], contiguous.

    The cache keeps one workspace for the attention, large enough for every call (workspace_bytes(): 22 or 43 MB at
    head_dim 64 or 128): `workspace`, a uint8 tensor that the caches of several layers may share, or a new one. A call
    that may overlap another one in time (another stream, a graph replayed beside it) passes one of its own.
    Keep the cache until its work on other streams than the one it was made on has ended, and as long as graphs replay it.

    Calls report into `status`, an int32 tensor that each call clears, or, without one, into a word of the cache that
    error() reads. Bit 0: positions of a sequence were outside the cache; bit 1: a wait on the device ran out, and the
    attention's results are not valid."""

    def __init__(self, n_kv_heads: int, head_dim: int, max_ctx: int, n_seqs: int = 1, fmt: int = TINFER_KV8_E4M3,
                 block: int = 64, device="cuda", buffers=None, workspace=None):
        import torch
        shape = tinfer_kv8(fmt, n_seqs, n_kv_heads, head_dim, max_ctx, block, *[16] * 4)  # (addresses that are not looked at)
        if lib().tinfer_kv8_attention_workspace(shape, n_kv_heads, 1) == 0:
            raise TinferError(TINFER_ERR_UNSUPPORTED, "Kv8Cache")
        codes = torch.Size((n_seqs, n_kv_heads, max_ctx, head_dim))
        scales = torch.Size((n_seqs, n_kv_heads, -(-max_ctx // max(1, block))))
        if buffers is None:
            device = torch.device(device)
            buffers = tuple(torch.zeros(codes, dtype=torch.uint8, device=device) for _ in range(2)) + tuple(
                torch.zeros(scales, dtype=torch.float32, device=device) for _ in range(2))
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = buffers
        self.device = self.k_codes.device
        if self.device.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        for what, t, dt, shape in zip(("k_codes", "v_codes", "k_scales", "v_scales"), buffers,
                                      (torch.uint8, torch.uint8, torch.float32, torch.float32),
                                      (codes, codes, scales, scales)):
            _on(what, t, self.device, dt, shape)
            if not t.is_contiguous():
                raise ValueError(f"{what} is not contiguous")
        self.n_seqs, self.n_kv_heads, self.head_dim, self.max_ctx = n_seqs, n_kv_heads, head_dim, max_ctx
        self._int32, self._uint8 = torch.int32, torch.uint8
        self.c, self._kept = (tinfer_kv8(f, n_seqs, n_kv_heads, head_dim, max_ctx, block, *(t.data_ptr() for t in buffers))
                              for f in (fmt, fmt | TINFER_KV8_KEEP_STATUS))
        need = self.workspace_bytes(n_kv_heads, 1)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._workspace = self._check_workspace(workspace)
        self._errors = torch.zeros(1, dtype=torch.int32, device=self.device)
        if not torch.cuda.is_current_stream_capturing():
            # calls may come on any stream: the zeros, and what the current stream still does with memory that is the
            # workspace now, come before them
            torch.cuda.current_stream(self.device).synchronize()

    def _rows(self, what, t, heads=None, tokens=None) -> tinfer_rows:
        s = t.shape
        if (len(s) != 4 or s[0] != self.n_seqs or s[3] != self.head_dim or (heads is not None and s[2] != heads)
                or (tokens is not None and s[1] != tokens)):
            raise ValueError(f"{what}: rows [{self.n_seqs}, n_tokens, heads, {self.head_dim}] are wanted, got {tuple(s)}")
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, not on {self.device}")
        st = t.stride()
        if st[3] != 1:
            raise ValueError(f"{what}: the elements of a row are not contiguous")
        return tinfer_rows(t.data_ptr(), _dtype(t), st[0], st[1], st[2])

    def _ints(self, what, t, n):
        """Address of an int32 argument of n values (None: no argument)."""
        if t is None:
            return None
        if t.dtype != self._int32 or t.numel() != n or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{what}: a contiguous int32 tensor of {n} on {self.device} is wanted")
        return t.data_ptr()

    def _status(self, status):
        """The cache's structure and the address of the status word of a call."""
        return (self._kept, self._errors.data_ptr()) if status is None else (self.c, self._ints("status", status, 1))

    def error(self) -> int:
        """Status bits of all calls without a `status` of their own since the last error(). Waits for the device."""
        import torch
        torch.cuda.synchronize(self.device)
        bits = int(self._errors)
        if bits:
            self._errors.zero_()
            torch.cuda.synchronize(self.device)
        return bits

    def append(self, k, v, pos, counts=None, rope_theta: float = 0.0, status=None, stream=None) -> None:
        """Quantises rows k and v into the cache at pos (keys rotated first; rope_theta 0: they already are)."""
        kr, vr = self._rows("k", k, self.n_kv_heads), self._rows("v", v, self.n_kv_heads, k.shape[1])
        c, word = self._status(status)
        _call("tinfer_op_kv8_append", lib().tinfer_op_kv8_append,
              (c, kr, vr, k.shape[1], self._ints("pos", pos, self.n_seqs), self._ints("counts", counts, self.n_seqs),
               rope_theta, word), self.device, stream)

    def read(self, n_tokens: int, pos, counts=None, out=None, dtype=None, status=None, stream=None):
        """Reads n_tokens tokens of each sequence from pos on back into rows (k, v): `out`, or new ones of dtype
        (bfloat16 when None), zero where a sequence has fewer tokens."""
        import torch
        if out is None:
            with _making(stream, self.device):
                out = tuple(torch.zeros((self.n_seqs, n_tokens, self.n_kv_heads, self.head_dim),
                                        dtype=dtype or torch.bfloat16, device=self.device) for _ in range(2))
        kr, vr = (self._rows(what, t, self.n_kv_heads, n_tokens) for what, t in zip(("k", "v"), out))
        c, word = self._status(status)
        _call("tinfer_op_kv8_read", lib().tinfer_op_kv8_read,
              (c, n_tokens, self._ints("pos", pos, self.n_seqs), self._ints("counts", counts, self.n_seqs), kr, vr, word),
              self.device, stream)
        return out

    def workspace_bytes(self, n_heads: int | None = None, n_tokens: int = 1) -> int:
        return lib().tinfer_kv8_attention_workspace(self.c, n_heads or self.n_kv_heads, n_tokens)

    def _check_workspace(self, t):
        if t.dtype != self._uint8 or t.device != self.device or not t.is_contiguous():
            raise ValueError("workspace: a contiguous uint8 tensor on the cache's device is wanted")
        return t

    def attention(self, q, pos, counts=None, rope_theta: float = 0.0, out=None, lse=None, workspace=None, status=None,
                  stream=None):
        """Attention of the query rows q over the cache: token i of sequence s attends to positions
        [0, pos[s] + i]. Returns `out` (rows like q; a new tensor, zero where a sequence has fewer tokens, when None)."""
        qr = self._rows("q", q)
        n_tokens, n_heads = q.shape[1], q.shape[2]
        if out is None:
            with _making(stream, self.device):
                out = q.new_zeros(q.shape)
        orow = self._rows("out", out, n_heads, n_tokens)
        if lse is not None and (lse.dtype != self.k_scales.dtype or lse.shape != q.shape[:3] or lse.device != self.device
                                or not lse.is_contiguous()):
            raise ValueError("lse: a contiguous float32 tensor [n_seqs, n_tokens, n_heads] is wanted")
        workspace = self._workspace if workspace is None else self._check_workspace(workspace)
        c, word = self._status(status)
        _call("tinfer_op_kv8_attention", lib().tinfer_op_kv8_attention,
              (c, n_heads, n_tokens, qr, self._ints("pos", pos, self.n_seqs), self._ints("counts", counts, self.n_seqs),
               rope_theta, orow, _ptr(lse), workspace.data_ptr(), workspace.numel(), word), self.device, stream)
        return out


def logprobs(logits, targets=None, top_k: int = 0, stream=None):
    """(logp, entropy, top_ids, top_logp) of the rows of logits [rows, vocab] (tinfer_op_logprobs): the log
    probability of each row's target token, the row's entropy, and its top_k likeliest tokens with theirs. logp
    is None without targets, the last two are None when top_k is 0."""
    import torch
    if logits.dim() != 2 or logits.stride(1) != 1 or logits.device.type != "cuda":
        raise ValueError("logits: [rows, vocab] on a CUDA device with contiguous rows is wanted")
    rows, vocab = logits.shape
    dev, dtype = logits.device, _dtype(logits)
    if targets is not None and (targets.dtype != torch.int32 or targets.shape != (rows,) or targets.device != dev
                                or not targets.is_contiguous()):
        raise ValueError(f"targets: a contiguous int32 tensor [{rows}] on {dev} is wanted")
    with _making(stream, dev):
        logp = torch.empty(rows, dtype=torch.float32, device=dev) if targets is not None else None
        entropy = torch.empty(rows, dtype=torch.float32, device=dev)
        ids = torch.empty((rows, top_k), dtype=torch.int32, device=dev) if top_k > 0 else None
        top = torch.empty((rows, top_k), dtype=torch.float32, device=dev) if top_k > 0 else None
    if rows == 0 and 0 <= top_k <= 32:
        return logp, entropy, ids, top  # nothing to launch
    _call("tinfer_op_logprobs", lib().tinfer_op_logprobs,
          (rows, vocab, dtype, logits.data_ptr(), logits.stride(0) if rows > 1 else vocab, _ptr(targets), top_k,
           _ptr(logp), entropy.data_ptr(), _ptr(ids), _ptr(top)), dev, stream)
    return logp, entropy, ids, top
