"""ctypes binding of libds4g.so (include/ds4g.h): argument marshalling only.

Device memory and streams come from PyTorch; pointers and sizes cross the C ABI.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libds4g.so")

F32, BF16 = 0, 1
OK, EINVAL, ECONTEXT, ETOKEN, ECUDA, ETIMEOUT, ESIZE, ENONFINITE = 0, -1, -2, -3, -4, -5, -6, -7
DEBUG = {"x": 0, "cqkv": 1, "q": 2, "attn": 3, "xmid": 4, "xn2": 5, "scores": 6, "h": 7,
         "hidden": 8, "prefill_x": 9, "status": 10, "prefill_layer_x": 11}


KERNEL_KINDS = ("qkv_a", "qkv_b", "attn", "wo", "router", "expert_gu", "expert_down", "lm_head",
                "p_embed", "p_norm", "p_qkv_a", "p_q_b", "p_kv_b", "p_attn", "p_wo", "p_router", "p_topk",
                "p_group", "p_gate_up", "p_shared_gu", "p_down", "p_shared_down", "p_combine")


class Ds4gError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {lib().ds4g_strerror(code).decode()} ({code})")
        self.code = code


class Config(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_layers", "hidden", "n_heads", "head_dim", "q_rank",
                                       "kv_rank", "window", "n_experts", "top_k",
                                       "expert_inter", "vocab")] + \
               [("rope_base", C.c_float), ("rms_eps", C.c_float), ("weight_dtype", C.c_int),
                ("kv_dtype", C.c_int), ("prefill_chunk", C.c_int), ("decode_kernel", C.c_int),
                ("prefill_kernel", C.c_int)]


LAYER_FIELDS = ("attn_norm", "wq_a", "wq_b", "wkv_a", "wk_b", "wv_b", "wo", "ffn_norm",
                "w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")


class LayerWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in LAYER_FIELDS]


class Weights(C.Structure):
    _fields_ = [("tok_embd", C.c_void_p), ("lm_head", C.c_void_p),
                ("layers", C.POINTER(LayerWeights))]


_lib = None


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(there is no fallback implementation)")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int, C.c_int64, C.c_size_t
        sig = {
            "ds4g_model_create": ([vp, vp, vp], i32),
            "ds4g_model_destroy": ([vp], None),
            "ds4g_session_bytes": ([vp, i32], sz),
            "ds4g_session_create": ([vp, i32, vp, sz, vp, vp], i32),
            "ds4g_session_destroy": ([vp], None),
            "ds4g_prefill": ([vp, vp, i32], i32),
            "ds4g_decode_step": ([vp, C.c_int32], i32),
            "ds4g_decode_layers": ([vp, C.c_int32], i32),
            "ds4g_sample_static": ([vp, i32, C.c_float, C.c_float, vp, vp], C.c_int32),
            "ds4g_session_hidden": ([vp], vp),
            "ds4g_session_common_prefix": ([vp, vp, i32], i32),
            "ds4g_session_truncate": ([vp, i32], i32),
            "ds4g_session_sync": ([vp, vp, i32, vp], i32),
            "ds4g_checkpoint_bytes": ([vp, i32], sz),
            "ds4g_session_save": ([vp, vp, sz], i32),
            "ds4g_session_load": ([vp, vp, sz], i32),
            "ds4g_session_rewrite_from_common": ([vp, vp, i32, i32], i32),
            "ds4g_session_len": ([vp], i32),
            "ds4g_session_logits": ([vp], vp),
            "ds4g_session_kv": ([vp, i32, vp, vp], i32),
            "ds4g_session_restore": ([vp, vp, i32], i32),
            "ds4g_session_router": ([vp, i32, vp, vp], i32),
            "ds4g_session_debug": ([vp, i32], vp),
            "ds4g_sample_workspace_bytes": ([i32], sz),
            "ds4g_session_launches": ([vp], C.c_uint64),
            "ds4g_session_status": ([vp], i32),
            "ds4g_session_set_trace": ([vp, vp, sz], i32),
            "ds4g_session_set_probe": ([vp, vp, i32, vp], i32),
            "ds4g_decode_layers_host": ([vp, C.c_int32, vp], i32),
            "ds4g_decode_sample": ([vp, C.c_int32, C.c_float, C.c_float, vp, vp, sz], C.c_int32),
            "ds4g_session_set_timing": ([vp, i32], i32),
            "ds4g_session_timing": ([vp, vp, vp, i32], i32),
            "ds4g_sample": ([vp, i32, C.c_float, C.c_float, vp, vp, sz, vp], C.c_int32),
            "ds4g_sample_u": ([vp, i32, C.c_float, C.c_float, C.c_uint32, vp, sz, vp], C.c_int32),
            "ds4g_sample_min_p": ([vp, i32, C.c_float, C.c_float, C.c_float, vp, vp, sz, vp], C.c_int32),
            "ds4g_sample_u_min_p": ([vp, i32, C.c_float, C.c_float, C.c_float, C.c_uint32, vp, sz, vp],
                                    C.c_int32),
            "ds4g_rope_fill": ([vp, i32, i32, C.c_float, vp], i32),
            "ds4g_paged_append": ([vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, i32, vp], i32),
            "ds4g_paged_attention_workspace_bytes": ([vp, vp, i32], sz),
            "ds4g_paged_attention": ([vp, vp, vp, i64, vp, i64, i32, i32, C.c_float, i32, vp, sz, vp], i32),
            "ds4g_paged_attention_status": ([vp, vp], i32),
            "ds4g_paged_append8": ([vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, i32, vp], i32),
            "ds4g_paged_attention8_workspace_bytes": ([vp, vp, i32], sz),
            "ds4g_paged_attention8": ([vp, vp, vp, i64, vp, i64, i32, i32, C.c_float, i32, vp, sz, vp], i32),
            "ds4g_paged_resize": ([vp, vp, i32, i32, vp, vp, i32, vp, vp, i32, vp], i32),
            "ds4g_edit_logits": ([vp, i64, i32, i32, vp, vp, i64, vp], i32),
            "ds4g_probs": ([vp, i64, i32, i32, C.c_float, vp, i64, vp], i32),
            "ds4g_verify_draft": ([vp, i64, i64, vp, i64, i64, vp, vp, vp, i32, i32, i32, vp, vp, vp], i32),
            "ds4g_strerror": ([i32], C.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(rc: int, what: str) -> int:
    if rc < 0:
        raise Ds4gError(rc, what)
    return rc


DECODE_AUTO, DECODE_STAGED = 0, 1
PREFILL_AUTO, PREFILL_SIMT, PREFILL_HILO = 0, 1, 2


def config_struct(shape, prefill_chunk: int = 0, decode_kernel: int = DECODE_AUTO,
                  prefill_kernel: int = PREFILL_AUTO) -> Config:
    c = Config()
    for n in ("n_layers", "hidden", "n_heads", "head_dim", "q_rank", "kv_rank", "window",
              "n_experts", "top_k", "expert_inter", "vocab"):
        setattr(c, n, int(getattr(shape, n)))
    c.rope_base = float(shape.rope_base)
    c.rms_eps = float(shape.rms_eps)
    c.weight_dtype = F32 if shape.weight_dtype == "f32" else BF16
    c.kv_dtype = F32 if shape.kv_dtype == "f32" else BF16
    c.prefill_chunk = int(prefill_chunk)
    c.decode_kernel = int(decode_kernel)
    c.prefill_kernel = int(prefill_kernel)
    return c


def session_bytes(shape, n_ctx: int, prefill_chunk: int = 0) -> int:
    c = config_struct(shape, prefill_chunk)
    return lib().ds4g_session_bytes(C.byref(c), n_ctx)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


class Model:
    """Weights are device tensors owned by the caller (kept referenced here)."""

    def __init__(self, shape, tok_embd: torch.Tensor, lm_head: torch.Tensor, layers: list,
                 prefill_chunk: int = 0, decode_kernel: int = DECODE_AUTO,
                 prefill_kernel: int = PREFILL_AUTO):
        self.shape = shape
        self.cfg = config_struct(shape, prefill_chunk, decode_kernel, prefill_kernel)
        self._keep = (tok_embd, lm_head, layers)
        arr = (LayerWeights * len(layers))()
        for i, w in enumerate(layers):
            for n in LAYER_FIELDS:
                setattr(arr[i], n, w[n].data_ptr())
        self._arr = arr
        wts = Weights(tok_embd.data_ptr(), lm_head.data_ptr(), arr)
        h = C.c_void_p()
        _check(lib().ds4g_model_create(C.byref(self.cfg), C.byref(wts), C.byref(h)),
               "ds4g_model_create")
        self.ptr = h.value

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.ds4g_model_destroy(self.ptr)
            self.ptr = None


class Session:
    def __init__(self, model: Model, n_ctx: int, stream=None, device="cuda"):
        self.model = model
        self.n_ctx = n_ctx
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        nbytes = lib().ds4g_session_bytes(C.byref(model.cfg), n_ctx)
        if nbytes == 0:
            raise Ds4gError(EINVAL, "ds4g_session_bytes")
        self.mem = torch.empty(nbytes, dtype=torch.uint8, device=device)
        h = C.c_void_p()
        _check(lib().ds4g_session_create(model.ptr, n_ctx, self.mem.data_ptr(), nbytes,
                                         _stream_ptr(self.stream), C.byref(h)),
               "ds4g_session_create")
        self.ptr = h.value

    def __del__(self):
        if getattr(self, "ptr", None) and _lib is not None:
            _lib.ds4g_session_destroy(self.ptr)
            self.ptr = None

    # -- calls ---------------------------------------------------------------
    def prefill(self, tokens) -> int:
        t = (C.c_int32 * len(tokens))(*[int(x) for x in tokens])
        return lib().ds4g_prefill(self.ptr, t, len(tokens))

    def decode(self, token: int) -> int:
        return lib().ds4g_decode_step(self.ptr, int(token))

    def decode_layers(self, token: int) -> int:
        """One token through every layer without the lm_head."""
        return lib().ds4g_decode_layers(self.ptr, int(token))

    def decode_layers_host(self, token: int, hidden_host: torch.Tensor) -> int:
        """ds4g_decode_layers with the final hidden state copied into hidden_host (a
        host float32 tensor of hidden elements, pinned for speed)."""
        assert hidden_host.dtype == torch.float32 and not hidden_host.is_cuda
        assert hidden_host.numel() == self.model.shape.hidden and hidden_host.is_contiguous()
        return lib().ds4g_decode_layers_host(self.ptr, int(token), hidden_host.data_ptr())

    def decode_sample(self, token: int, temperature: float, top_p: float, rng_state, ws: torch.Tensor):
        """ds4g_decode_sample: one decode step and the next token's draw; returns
        (token or negative code, new rng state)."""
        st = C.c_uint64(rng_state if rng_state is not None else 0)
        tok = lib().ds4g_decode_sample(self.ptr, int(token), float(temperature), float(top_p), C.byref(st),
                                       ws.data_ptr(), ws.numel() * ws.element_size())
        return tok, st.value

    def hidden(self) -> torch.Tensor:
        return self._view(lib().ds4g_session_hidden(self.ptr), self.model.shape.hidden,
                          torch.float32)

    def truncate(self, cp: int) -> int:
        return lib().ds4g_session_truncate(self.ptr, int(cp))

    def sync(self, tokens):
        """Bring the session to the prompt `tokens`: (status, tokens prefilled)."""
        t = (C.c_int32 * max(1, len(tokens)))(*[int(x) for x in tokens])
        n = C.c_int(0)
        rc = lib().ds4g_session_sync(self.ptr, t, len(tokens), C.byref(n))
        return rc, n.value

    def checkpoint_bytes(self) -> int:
        return int(lib().ds4g_checkpoint_bytes(C.byref(self.model.cfg), self.len))

    def save(self, buf: bytearray) -> int:
        """Write the session's checkpoint into the host buffer `buf`."""
        b = (C.c_char * len(buf)).from_buffer(buf)
        return lib().ds4g_session_save(self.ptr, b, len(buf))

    def load(self, buf) -> int:
        b = (C.c_char * len(buf)).from_buffer_copy(bytes(buf))
        return lib().ds4g_session_load(self.ptr, b, len(buf))

    def rewrite_from_common(self, tokens, common: int) -> int:
        t = (C.c_int32 * max(1, len(tokens)))(*[int(x) for x in tokens])
        return lib().ds4g_session_rewrite_from_common(self.ptr, t, len(tokens), int(common))

    def common_prefix(self, tokens) -> int:
        t = (C.c_int32 * len(tokens))(*[int(x) for x in tokens])
        return lib().ds4g_session_common_prefix(self.ptr, t, len(tokens))

    def restore(self, tokens) -> int:
        t = (C.c_int32 * len(tokens))(*[int(x) for x in tokens])
        return lib().ds4g_session_restore(self.ptr, t, len(tokens))

    @property
    def len(self) -> int:
        return lib().ds4g_session_len(self.ptr)

    # -- views of device buffers -----------------------------------------------
    def _view(self, ptr: int, n: int, dtype) -> torch.Tensor:
        off = ptr - self.mem.data_ptr()
        esz = torch.empty((), dtype=dtype).element_size()
        assert 0 <= off and off + n * esz <= self.mem.numel()
        return self.mem[off:off + n * esz].view(dtype)

    def logits(self) -> torch.Tensor:
        return self._view(lib().ds4g_session_logits(self.ptr), self.model.shape.vocab,
                          torch.float32)

    def debug(self, name: str, n: int) -> torch.Tensor:
        return self._view(lib().ds4g_session_debug(self.ptr, DEBUG[name]), n, torch.float32)

    def kv(self, layer: int):
        k, v = C.c_void_p(), C.c_void_p()
        _check(lib().ds4g_session_kv(self.ptr, layer, C.byref(k), C.byref(v)), "ds4g_session_kv")
        s = self.model.shape
        dt = torch.float32 if s.kv_dtype == "f32" else torch.bfloat16
        n = self.n_ctx * s.head_dim
        return (self._view(k.value, n, dt).view(self.n_ctx, s.head_dim),
                self._view(v.value, n, dt).view(self.n_ctx, s.head_dim))

    def set_trace(self, buf) -> None:
        """buf: a device tensor receiving per-CTA stage start times (or None)."""
        _check(lib().ds4g_session_set_trace(self.ptr, buf.data_ptr() if buf is not None else None,
                                            buf.numel() * buf.element_size() if buf is not None
                                            else 0), "ds4g_session_set_trace")

    def set_probe(self, positions) -> torch.Tensor | None:
        """Record the residual entering every layer (then the final hidden state) at
        the given session positions during later prefills and decode steps.  Returns
        the device buffer [n][L+1][H] (f32) the rows go to; an empty list stops it."""
        pos = (C.c_int32 * len(positions))(*[int(p) for p in positions])
        s = self.model.shape
        buf = torch.full((len(positions), s.n_layers + 1, s.hidden), float("nan"),
                         dtype=torch.float32, device="cuda") if len(positions) else None
        _check(lib().ds4g_session_set_probe(self.ptr, pos, len(positions),
                                            buf.data_ptr() if buf is not None else None),
               "ds4g_session_set_probe")
        self._probe = buf   # kept alive while the setting holds
        return buf

    def status(self) -> int:
        return lib().ds4g_session_status(self.ptr)

    @property
    def launches(self) -> int:
        return lib().ds4g_session_launches(self.ptr)

    def set_timing(self, on: bool) -> None:
        _check(lib().ds4g_session_set_timing(self.ptr, int(on)), "ds4g_session_set_timing")

    def timing(self):
        """{kernel kind: (total ms, launches)} since the last call (timing mode)."""
        n = len(KERNEL_KINDS)
        ms = (C.c_double * n)()
        cnt = (C.c_uint64 * n)()
        _check(lib().ds4g_session_timing(self.ptr, ms, cnt, n), "ds4g_session_timing")
        return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}

    def router(self, layer: int):
        K = self.model.shape.top_k
        ids = (C.c_int32 * K)()
        w = (C.c_float * K)()
        _check(lib().ds4g_session_router(self.ptr, layer, ids, w), "ds4g_session_router")
        return list(ids), list(w)


def sample_workspace_bytes(n_vocab: int) -> int:
    return lib().ds4g_sample_workspace_bytes(n_vocab)


def sample(logits: torch.Tensor, temperature: float, top_p: float, rng_state: int | None,
           workspace: torch.Tensor, stream=None, min_p: float = 0.0):
    """Returns (token, new_rng_state); min_p > 0 calls ds4g_sample_min_p."""
    st = C.c_uint64(rng_state or 0)
    if min_p > 0.0:
        tok = lib().ds4g_sample_min_p(logits.data_ptr(), logits.numel(), float(temperature),
                                      float(top_p), float(min_p), C.byref(st), workspace.data_ptr(),
                                      workspace.numel(), _stream_ptr(stream))
    else:
        tok = lib().ds4g_sample(logits.data_ptr(), logits.numel(), float(temperature), float(top_p),
                                C.byref(st), workspace.data_ptr(), workspace.numel(),
                                _stream_ptr(stream))
    return tok, st.value


def sample_static(logits: torch.Tensor, temperature: float, top_p: float,
                  rng_state: int | None, stream=None):
    """ds4g_sample_static: no workspace argument; returns (token, new_rng_state)."""
    st = C.c_uint64(rng_state or 0)
    tok = lib().ds4g_sample_static(logits.data_ptr(), logits.numel(), float(temperature),
                                   float(top_p), C.byref(st), _stream_ptr(stream))
    return tok, st.value


def sample_u(logits: torch.Tensor, temperature: float, top_p: float, u24: int,
             workspace: torch.Tensor, stream=None, min_p: float = 0.0) -> int:
    """Sample with a caller-given uniform draw u = u24 / 2^24."""
    if min_p > 0.0:
        return lib().ds4g_sample_u_min_p(logits.data_ptr(), logits.numel(), float(temperature),
                                         float(top_p), float(min_p), int(u24), workspace.data_ptr(),
                                         workspace.numel(), _stream_ptr(stream))
    return lib().ds4g_sample_u(logits.data_ptr(), logits.numel(), float(temperature),
                               float(top_p), int(u24), workspace.data_ptr(), workspace.numel(),
                               _stream_ptr(stream))


# ---------------------------------------------------------------- operators on device buffers

class PagedKVStruct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64),
                ("slot_stride", C.c_int64), ("head_stride", C.c_int64), ("n_pages", C.c_int),
                ("page_size", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("dtype", C.c_int)]


class PagedKV8Struct(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("page_stride", C.c_int64), ("slot_stride", C.c_int64), ("head_stride", C.c_int64),
                ("scale_stride", C.c_int64), ("n_pages", C.c_int), ("page_size", C.c_int),
                ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("block", C.c_int)]


class PagePoolStruct(C.Structure):
    _fields_ = [("free_pages", C.c_void_p), ("n_free", C.c_void_p), ("capacity", C.c_int), ("page_size", C.c_int)]


class LogitEditsStruct(C.Structure):
    _fields_ = [("history", C.c_void_p), ("n_history", C.c_void_p), ("n_prompt", C.c_void_p),
                ("history_stride", C.c_int64), ("repetition", C.c_void_p), ("frequency", C.c_void_p),
                ("presence", C.c_void_p), ("bias_ids", C.c_void_p), ("n_bias", C.c_void_p), ("bias", C.c_void_p),
                ("bias_stride", C.c_int64), ("allowed", C.c_void_p), ("allowed_stride", C.c_int64),
                ("max_history", C.c_int), ("max_bias", C.c_int)]


class PagedBatchStruct(C.Structure):
    _fields_ = [("table", C.c_void_p), ("length", C.c_void_p), ("start", C.c_void_p),
                ("n_seqs", C.c_int), ("n_tokens", C.c_int), ("max_new", C.c_int),
                ("width", C.c_int), ("table_stride", C.c_int)]


class RopeStruct(C.Structure):
    _fields_ = [("cs", C.c_void_p), ("n_pos", C.c_int), ("rot_dim", C.c_int)]


_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _int32(n: int) -> int:
    """n within a C int, below 0 as 0 (ctypes would take its low 32 bits)."""
    return min(max(n, 0), 0x7fffffff)


def _require(ok: bool, what: str) -> None:
    if not ok:
        raise Ds4gError(EINVAL, what)


# The current stream's handle without building a Stream object (3 us of a small call's 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, index: int, stream, *args) -> None:
    """One call of the library on CUDA device `index`, on `stream` (None: that device's
    current stream)."""
    if index < 0:   # a CPU tensor
        raise Ds4gError(EINVAL, name)
    f = getattr(_lib or lib(), name)
    st = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        rc = f(*args, st)
    else:
        with torch.cuda.device(index):
            rc = f(*args, st)
    if rc < 0:
        raise Ds4gError(rc, name)


class PagedKV:
    """The paged K/V cache of one layer (ds4g_paged_kv): k and v [n_pages][page_size]
    [n_kv_heads][head_dim], of equal strides, the last dimension adjacent."""

    calls = ("ds4g_paged_append", "ds4g_paged_attention", "ds4g_paged_attention_workspace_bytes")

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _require(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.stride(3) == 1 and
                 k.dtype == v.dtype and k.dtype in _DTYPES and k.device == v.device, "PagedKV")
        self.k, self.v, self.index = k, v, k.get_device()
        n, p, h, d = k.shape
        self.n_kv_heads, self.head_dim = h, d
        self.struct = PagedKVStruct(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                                    n, p, h, d, _DTYPES[k.dtype])
        self.ref = C.addressof(self.struct)


class PagedKV8:
    """The paged K/V cache of one layer in 8 bits (ds4g_paged_kv8): codes k and v
    (torch.float8_e4m3fn) as PagedKV's, and k_scale, v_scale (f32) [n_pages][blocks][n_kv_heads]
    of equal strides, the last two dimensions adjacent; a scale is that of page_size / blocks
    slots.  paged_append and paged_attention take either cache."""

    calls = ("ds4g_paged_append8", "ds4g_paged_attention8", "ds4g_paged_attention8_workspace_bytes")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        _require(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride() and k.stride(3) == 1 and
                 k.dtype == v.dtype == torch.float8_e4m3fn and k_scale.dim() == 3 and k_scale.shape == v_scale.shape and
                 k_scale.stride() == v_scale.stride() and k_scale.dtype == v_scale.dtype == torch.float32 and
                 k.device == v.device == k_scale.device == v_scale.device, "PagedKV8")
        n, p, h, d = k.shape
        blocks, s = k_scale.shape[1], k_scale.stride()
        _require(k_scale.shape[0] == n and k_scale.shape[2] == h and blocks > 0 and p % blocks == 0 and
                 (h <= 1 or s[2] == 1) and (blocks <= 1 or s[1] == h), "PagedKV8")
        self.k, self.v, self.k_scale, self.v_scale, self.index = k, v, k_scale, v_scale, k.get_device()
        self.n_kv_heads, self.head_dim, self.block = h, d, p // blocks
        self.struct = PagedKV8Struct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0),
                                     k.stride(1), k.stride(2), s[0] if n > 1 else blocks * h, n, p, h, d, self.block)
        self.ref = C.addressof(self.struct)


class PagedBatch:
    """The sequences of a call (ds4g_paged_batch): int32 device tensors table [n_seqs]
    [width], length [n_seqs] and start [n_seqs + 1] (None: one new token each).  The
    tensors are kept, and read by each call as they then are; max_new bounds a sequence's
    new tokens.  A batch has one owner thread, as a session has."""

    def __init__(self, table: torch.Tensor, length: torch.Tensor, start: torch.Tensor | None = None,
                 max_new: int = 1):
        n = length.numel()
        _require(table.dim() == 2 and table.shape[0] == n and table.dtype == torch.int32 and
                 (table.shape[1] <= 1 or table.stride(1) == 1) and
                 (n <= 1 or table.stride(0) >= table.shape[1]) and length.dtype == torch.int32 and
                 length.is_contiguous() and table.device == length.device, "PagedBatch")
        _require(start is None or (start.dtype == torch.int32 and start.numel() == n + 1 and
                                   start.is_contiguous() and start.device == length.device), "PagedBatch")
        self.table, self.length, self.start, self.index = table, length, start, length.get_device()
        width = table.shape[1]
        self.struct = PagedBatchStruct(table.data_ptr(), length.data_ptr(),
                                       start.data_ptr() if start is not None else None, n, n, _int32(max_new),
                                       width, table.stride(0) if n > 1 else width)
        self.ref = C.addressof(self.struct)


class Rope:
    """Rotation table (ds4g_rope): cs [n_pos][rot_dim / 2][2] f32, (cos, sin) of every pair."""

    def __init__(self, cs: torch.Tensor):
        _require(cs.dim() == 3 and cs.shape[2] == 2 and cs.dtype == torch.float32 and cs.is_contiguous(), "Rope")
        self.cs, self.index = cs, cs.get_device()
        self.struct = RopeStruct(cs.data_ptr(), cs.shape[0], 2 * cs.shape[1])
        self.ref = C.addressof(self.struct)

    @classmethod
    def fill(cls, n_pos: int, rot_dim: int, base: float = 10000.0, device="cuda", stream=None) -> "Rope":
        """A table filled by ds4g_rope_fill."""
        cs = torch.empty(n_pos, rot_dim // 2, 2, dtype=torch.float32, device=device)
        _call("ds4g_rope_fill", cs.get_device(), stream, cs.data_ptr(), n_pos, rot_dim, float(base))
        return cls(cs)


def _rows(t: torch.Tensor, n: int, heads: int, dim: int, dtype, index: int, what: str) -> int:
    """Token stride of t, a token tensor [n][heads][dim] of `dtype`, heads and dims adjacent."""
    if t.shape == (n, heads, dim) and t.dtype is dtype and t.get_device() == index:
        s = t.stride()
        if s[2] == 1 and (s[1] == dim or heads == 1):
            return s[0] if n > 1 else heads * dim
    raise Ds4gError(EINVAL, what)


def _tokens(batch: PagedBatch, t: torch.Tensor) -> int:
    """Rows of a call's token tensors: as many as there are sequences without starts, else t's."""
    if batch.start is None:
        return batch.struct.n_tokens
    batch.struct.n_tokens = n = t.shape[0]
    return n


def paged_append(kv: PagedKV | PagedKV8, batch: PagedBatch, k: torch.Tensor, v: torch.Tensor, rope: Rope | None = None,
                 q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, stream=None) -> None:
    """ds4g_paged_append, ds4g_paged_append8: k, v [n_tokens][n_kv_heads][head_dim] into the cache's pages, the
    keys rotated by `rope`; q [n_tokens][n_heads][head_dim] rotated into q_out (which may
    be q)."""
    n, h, d, dt, index, what = _tokens(batch, k), kv.n_kv_heads, kv.head_dim, k.dtype, batch.index, "paged_append"
    _require(dt in _DTYPES and kv.index == index and (rope is None or rope.index == index) and
             (q is None) == (q_out is None), what)
    ks, vs = _rows(k, n, h, d, dt, index, what), _rows(v, n, h, d, dt, index, what)
    rp = rope.ref if rope is not None else None
    if q is None:
        _call(kv.calls[0], index, stream, kv.ref, batch.ref, k.data_ptr(), ks, v.data_ptr(), vs, rp, None, 0,
              None, 0, 0, _DTYPES[dt])
        return
    _require(q.dim() == 3, what)
    heads = q.shape[1]
    _call(kv.calls[0], index, stream, kv.ref, batch.ref, k.data_ptr(), ks, v.data_ptr(), vs, rp, q.data_ptr(),
          _rows(q, n, heads, d, dt, index, what), q_out.data_ptr(), _rows(q_out, n, heads, d, dt, index, what), heads,
          _DTYPES[dt])


def paged_attention_workspace_bytes(kv: PagedKV | PagedKV8, batch: PagedBatch, n_heads: int) -> int:
    return getattr(lib(), kv.calls[2])(kv.ref, batch.ref, n_heads)


def paged_attention(kv: PagedKV | PagedKV8, batch: PagedBatch, q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                    scale: float = 0.0, window: int = 0, stream=None) -> None:
    """ds4g_paged_attention, ds4g_paged_attention8: q and out [n_tokens][n_heads][head_dim]; scale 0: 1 /
    sqrt(head_dim); window 0: every position up to the token's own."""
    _require(q.dim() == 3 and q.dtype in _DTYPES and kv.index == batch.index == workspace.get_device() and
             workspace.is_contiguous(), "paged_attention")
    n, d, dt, heads, index = _tokens(batch, q), kv.head_dim, q.dtype, q.shape[1], batch.index
    _call(kv.calls[1], index, stream, kv.ref, batch.ref, q.data_ptr(),
          _rows(q, n, heads, d, dt, index, "paged_attention"), out.data_ptr(),
          _rows(out, n, heads, d, dt, index, "paged_attention"), heads, _DTYPES[dt], scale, _int32(window),
          workspace.data_ptr(), workspace.nbytes)


_STATUS_BYTES = 4 * 320   # of a workspace: what ds4g_paged_attention_status reads


def paged_attention_status(workspace: torch.Tensor, stream=None) -> int:
    """ds4g_paged_attention_status: OK, or once ETIMEOUT after calls on the workspace in which a
    wait gave up (synchronises)."""
    index = workspace.get_device()
    _require(index >= 0 and workspace.is_contiguous() and workspace.nbytes >= _STATUS_BYTES, "paged_attention_status")
    with torch.cuda.device(index):   # (a null stream is the current device's)
        return lib().ds4g_paged_attention_status(workspace.data_ptr(),
                                                 _raw_stream(index) if stream is None else stream.cuda_stream)


class PagePool:
    """Pages that no sequence holds (ds4g_page_pool): int32 device tensors free [capacity], a stack, and
    n_free [1], its height."""

    def __init__(self, free: torch.Tensor, n_free: torch.Tensor, page_size: int):
        _require(free.dim() == 1 and free.dtype == n_free.dtype == torch.int32 and free.is_contiguous() and
                 n_free.numel() == 1 and free.device == n_free.device and 0 < page_size < 2 ** 31, "PagePool")
        self.free, self.n_free, self.page_size, self.index = free, n_free, page_size, free.get_device()
        self.struct = PagePoolStruct(free.data_ptr(), n_free.data_ptr(), free.numel(), page_size)
        self.ref = C.addressof(self.struct)


def paged_resize(pool: PagePool, batch: PagedBatch, want: torch.Tensor, slots: torch.Tensor | None = None,
                 max_tokens: int | None = None, stream=None) -> None:
    """ds4g_paged_resize: the batch's lengths to want [n_seqs] (int32), its table and start with them, pages
    from and to the pool; slots (int64, or None) gets the slot of every new token.  max_tokens: the new
    tokens of all sequences at most (slots' size; without slots, any number)."""
    s, n, what = batch.struct, batch.struct.n_seqs, "paged_resize"
    _require(batch.start is not None and want.dtype == torch.int32 and want.numel() == n and want.is_contiguous() and
             pool.index == batch.index == want.get_device() and (n == 0 or want.data_ptr() != s.length), what)
    most = 2 ** 31 - 1 if max_tokens is None else _int32(max_tokens)
    if slots is not None:
        _require(slots.dtype == torch.int64 and slots.dim() == 1 and slots.is_contiguous() and
                 slots.get_device() == batch.index and (max_tokens is None or max_tokens <= slots.numel()), what)
        most = min(most, slots.numel())
    _call("ds4g_paged_resize", batch.index, stream, pool.ref, s.table, s.width, s.table_stride, s.length,
          want.data_ptr(), n, s.start, slots.data_ptr() if slots is not None else None, most)


class LogitEdits:
    """What edit_logits does to each row (ds4g_logit_edits).  Int32 device tensors history [n_rows]
    [max_history], n_history and n_prompt [n_rows], bias_ids [n_rows][max_bias], n_bias [n_rows], allowed [n_rows]
    or [1][at least n_vocab / 32 words]; f32 ones repetition, frequency, presence [n_rows], bias [n_rows]
    [max_bias].  Each may be None; the tensors are kept, and read by each call as they then are."""

    def __init__(self, history=None, n_history=None, n_prompt=None, repetition=None, frequency=None, presence=None,
                 bias_ids=None, bias=None, n_bias=None, allowed=None):
        what, i32, f32 = "LogitEdits", torch.int32, torch.float32
        self.tensors = (history, n_history, n_prompt, repetition, frequency, presence, bias_ids, bias, n_bias, allowed)
        there = [t for t in self.tensors if t is not None]
        self.index = there[0].get_device() if there else None
        _require(all(t.get_device() == self.index for t in there), what)
        rows = []

        def table(t, dtype):   # rows of adjacent values
            _require(t.dim() == 2 and t.dtype == dtype and (t.shape[1] <= 1 or t.stride(1) == 1) and
                     (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]), what)
            rows.append(t.shape[0])
            return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1], t.shape[1]

        def column(t, dtype):
            if t is None:
                return None
            _require(t.dim() == 1 and t.dtype == dtype and t.is_contiguous(), what)
            rows.append(t.shape[0])
            return t.data_ptr()

        s = self.struct = LogitEditsStruct()
        if history is not None:
            s.history, s.history_stride, s.max_history = table(history, i32)
        else:
            _require(all(t is None for t in (n_history, n_prompt, repetition, frequency, presence)), what)
        _require((bias_ids is None) == (bias is None) and (bias is not None or n_bias is None), what)
        if bias is not None:
            s.bias_ids, s.bias_stride, s.max_bias = table(bias_ids, i32)
            at, stride, most = table(bias, f32)
            _require(stride == s.bias_stride and most == s.max_bias, what)
            s.bias = at
        s.n_history, s.n_prompt, s.n_bias = column(n_history, i32), column(n_prompt, i32), column(n_bias, i32)
        s.repetition, s.frequency, s.presence = (column(t, f32) for t in (repetition, frequency, presence))
        self.words = None   # of a row of the mask
        if allowed is not None:
            one = allowed.dim() == 2 and allowed.shape[0] == 1
            s.allowed, s.allowed_stride, self.words = table(allowed, i32)
            if one:   # any number of rows
                s.allowed_stride = 0
                rows.pop()
        _require(len(set(rows)) <= 1, what)
        self.rows = rows[0] if rows else None   # None: any number
        self.ref = C.addressof(s)


def edit_logits(logits: torch.Tensor, out: torch.Tensor, edits: LogitEdits, stream=None) -> None:
    """ds4g_edit_logits: rows of f32 logits [n_rows][n_vocab] into out (which may be logits)."""
    shape, zs, ps, index = logits.shape, logits.stride(), out.stride(), logits.get_device()
    _require(len(shape) == 2 and shape == out.shape and logits.dtype is torch.float32 and out.dtype is torch.float32 and
             index == out.get_device() and (shape[1] <= 1 or zs[1] == ps[1] == 1) and
             (edits.index is None or edits.index == index), "edit_logits")
    n, v = shape
    _require((edits.rows is None or edits.rows == n) and (edits.words is None or 32 * edits.words >= v), "edit_logits")
    _call("ds4g_edit_logits", index, stream, logits.data_ptr(), zs[0] if n > 1 else v, n, v, edits.ref,
          out.data_ptr(), ps[0] if n > 1 else v)


def probs(logits: torch.Tensor, temperature: float, out: torch.Tensor, stream=None) -> None:
    """ds4g_probs: rows of f32 logits [n_rows][n_vocab] to probabilities (out may be logits)."""
    shape, zs, ps, index = logits.shape, logits.stride(), out.stride(), logits.get_device()
    _require(len(shape) == 2 and shape == out.shape and logits.dtype is torch.float32 and out.dtype is torch.float32 and
             index == out.get_device() and (shape[1] <= 1 or zs[1] == ps[1] == 1), "probs")
    n, v = shape
    _call("ds4g_probs", index, stream, logits.data_ptr(), zs[0] if n > 1 else v, n, v, float(temperature),
          out.data_ptr(), ps[0] if n > 1 else v)


def verify_draft(p: torch.Tensor, q: torch.Tensor | None, drafts: torch.Tensor, u24: torch.Tensor,
                 accepted: torch.Tensor, tokens: torch.Tensor, n_drafts: torch.Tensor | None = None,
                 stream=None) -> None:
    """ds4g_verify_draft: p [n_seqs][max_drafts + 1][n_vocab] and q [n_seqs][max_drafts][n_vocab]
    (or None) f32; drafts [n_seqs][max_drafts], u24 [n_seqs][max_drafts + 1], accepted [n_seqs], tokens
    [n_seqs][max_drafts + 1] and n_drafts [n_seqs] (or None) int32."""
    shape, what, index, i32 = p.shape, "verify_draft", p.get_device(), torch.int32
    _require(len(shape) == 3 and p.dtype is torch.float32, what)
    b, d1, v = shape
    d = d1 - 1
    per_draft, per_number = (b, d), (b, d1)
    if not (drafts.dtype is i32 and drafts.shape == per_draft and drafts.is_contiguous() and
            u24.dtype is i32 and u24.shape == per_number and u24.is_contiguous() and
            tokens.dtype is i32 and tokens.shape == per_number and tokens.is_contiguous() and
            accepted.dtype is i32 and accepted.shape == (b,) and accepted.is_contiguous() and
            drafts.get_device() == u24.get_device() == tokens.get_device() == accepted.get_device() == index):
        raise Ds4gError(EINVAL, what)
    n_ptr = None
    if n_drafts is not None:
        _require(n_drafts.dtype is i32 and n_drafts.shape == (b,) and n_drafts.is_contiguous() and
                 n_drafts.get_device() == index, what)
        n_ptr = n_drafts.data_ptr()

    def strides(t, rows):   # of a sequence and of a position; a dimension of one element has any stride
        s = t.stride()
        if not (v <= 1 or s[2] == 1):
            raise Ds4gError(EINVAL, what)
        pos = s[1] if rows > 1 else v
        return (s[0] if b > 1 else max(v, rows * pos)), pos

    ps, pp = strides(p, d1)
    qa, qs, qp = None, 0, 0
    if q is not None:
        _require(q.dtype is torch.float32 and q.shape == (b, d, v) and q.get_device() == index, what)
        qa = q.data_ptr()
        qs, qp = strides(q, d)
    _call("ds4g_verify_draft", index, stream, p.data_ptr(), ps, pp, qa, qs, qp, drafts.data_ptr(), n_ptr,
          u24.data_ptr(), b, d, v, accepted.data_ptr(), tokens.data_ptr())
