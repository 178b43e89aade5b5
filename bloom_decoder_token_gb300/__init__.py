"""Python binding of the GB300 BLOOM decode engine (``libbloom.so``).

Argument marshalling only: every step of the path runs in the CUDA library
behind the C ABI of ``include/bloom.h``.  PyTorch supplies device memory and
streams.  There is no CPU fallback: if the library is missing, every entry
point raises.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import NamedTuple, Optional

import torch

from . import synth

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbloom.so")
_lib = None

BLOOM_OK = 0
STATUS = {0: "OK", 1: "E_INVALID", 2: "E_UNSUPPORTED", 3: "E_OOM", 4: "E_CAPACITY",
          5: "E_CUDA", 6: "E_DEVICE_FLAG"}
EPI_STORE, EPI_GELU, EPI_RESID = 0, 1, 2
FLAG_NO_GRAPH = 1
FLAG_NO_PDL = 2
FLAG_NO_LN_FUSION = 4
FLAG_NO_TC_GEMM = 8

OPS = ("embed", "layernorm", "qkv", "attn", "dense", "up", "down", "head")
KERNELS = ("embed_kernel", "layernorm_kernel", "linear_kernel", "gemv_tc_kernel",
           "gemm_tc_kernel", "attn_decode_kernel", "attn_prefill_kernel")

P = C.c_void_p
I32 = C.c_int32


class BloomError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"bloom {STATUS.get(status, status)}: {msg}")
        self.status = status


class Config(C.Structure):
    _fields_ = [("n_layer", I32), ("hidden", I32), ("n_head", I32), ("ffn", I32),
                ("vocab", I32), ("ln_eps", C.c_float), ("weight_dtype", I32),
                ("max_batch", I32), ("max_tokens", I32), ("max_seq", I32), ("flags", I32),
                ("wait_us", I32)]


class Linear(C.Structure):
    _fields_ = [("w", P), ("scale", P), ("bias", P)]


class LayerWeights(C.Structure):
    _fields_ = [("ln1_g", P), ("ln1_b", P), ("qkv", Linear), ("o", Linear), ("ln2_g", P),
                ("ln2_b", P), ("up", Linear), ("down", Linear)]


class WeightsC(C.Structure):
    _fields_ = [("word_emb", P), ("emb_ln_g", P), ("emb_ln_b", P), ("lnf_g", P), ("lnf_b", P),
                ("layers", C.POINTER(LayerWeights))]


MAX_BATCH = 256


class KVC(C.Structure):
    _fields_ = [("buf", P), ("bytes", C.c_size_t), ("batch", I32), ("max_seq", I32),
                ("len", I32), ("row_len", I32 * MAX_BATCH), ("row_active", C.c_uint8 * MAX_BATCH),
                ("host_buf", P), ("host_bytes", C.c_size_t), ("offload_from", I32)]


class W4C(C.Structure):
    _fields_ = [("tiles", P), ("n", I32), ("k", I32), ("group", I32)]


class KV8C(C.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("codes", I32),
                ("batch", I32), ("n_kv", I32), ("max_seq", I32), ("d", I32)]


_SIGS = {
    "bloom_kv_bytes": (C.c_size_t, [C.POINTER(Config), I32, I32]),
    "bloom_create": (I32, [C.POINTER(Config), C.POINTER(WeightsC), C.POINTER(P)]),
    "bloom_kv_init": (I32, [P, C.POINTER(KVC), P, C.c_size_t, I32, I32, P]),
    "bloom_kv_bytes_offload": (I32, [C.POINTER(Config), I32, I32, I32, C.POINTER(C.c_size_t),
                                     C.POINTER(C.c_size_t)]),
    "bloom_kv_init_offload": (I32, [P, C.POINTER(KVC), P, C.c_size_t, P, C.c_size_t, I32, I32, I32,
                                    P]),
    "bloom_prefill": (I32, [P, C.POINTER(KVC), P, P, I32, I32, P, P, P]),
    "bloom_decode_step": (I32, [P, C.POINTER(KVC), P, P, P, P]),
    "bloom_decode_step_sampled": (I32, [P, C.POINTER(KVC), P, P, P, P, P, P, P]),
    "bloom_kv_admit": (I32, [P, C.POINTER(KVC), P, I32, P, P, I32, P, P, P]),
    "bloom_kv_retire": (I32, [P, C.POINTER(KVC), P, I32, P]),
    "bloom_generate": (I32, [P, C.POINTER(KVC), P, P, I32, I32, I32, P, P]),
    "bloom_check_device": (I32, [P, P]),
    "bloom_decode_profile": (I32, [P, C.POINTER(KVC), P, P, P, P, I32, P, P]),
    "bloom_destroy": (I32, [P]),
    "bloom_last_error": (C.c_char_p, []),
    "bloom_decode_launches": (I32, [P, I32]),
    "bloom_layer_decode": (I32, [P, C.POINTER(KVC), I32, P, P]),
    "bloom_kv_set_prompt": (I32, [P, C.POINTER(KVC), P, I32, I32, P]),
    "bloom_layer_prefill": (I32, [P, C.POINTER(KVC), I32, P, I32, I32, P]),
    "bloom_head": (I32, [P, P, I32, P, P, P]),
    "bloom_lm_head": (I32, [P, P, I32, P, P, P]),
    "bloom_embed": (I32, [P, P, I32, P, P]),
    "bloom_op_layernorm": (I32, [P, P, P, I32, I32, C.c_float, P, P]),
    "bloom_op_linear": (I32, [C.POINTER(Linear), I32, P, I32, I32, I32, I32, P, P]),
    "bloom_op_gemm": (I32, [C.POINTER(Linear), P, I32, I32, I32, I32, P, P]),
    "bloom_op_linear_tc": (I32, [C.POINTER(Linear), I32, P, I32, I32, I32, I32, P, P]),
    "bloom_op_attn_decode": (I32, [P, P, P, P, P, I32, I32, I32, I32, I32, I32, P, P]),
    "bloom_op_lmhead_argmax": (I32, [P, P, I32, I32, I32, P, P, P]),
    "bloom_op_sample": (I32, [P, I32, I32, C.c_int64, P, P, P, P, P]),
    "bloom_op_sample_filtered": (I32, [P, I32, I32, C.c_int64, P, P, P, P, P, I32, P, P]),
    "bloom_op_logprobs": (I32, [P, I32, I32, C.c_int64, P, I32, P, P, I32, P, P, P]),
    "bloom_op_kv8_write": (I32, [P, P, P, P, P, I32, P, P, P, P, P]),
    "bloom_op_kv8_read": (I32, [P, P, P, P, P, I32, P, P, P, P]),
    "bloom_op_attn_decode_kv8": (I32, [P, P, P, P, P, I32, I32, P, P, C.c_size_t, P, P]),
    "bloom_op_attn_decode_kv8_workspace": (C.c_size_t, [P, I32, I32]),
    "bloom_op_attn_decode_kv8_wait_us": (I32, [I32]),
    "bloom_w4_bytes": (C.c_size_t, [I32, I32, I32]),
    "bloom_op_w4_quantize": (I32, [P, C.c_int64, P, P]),
    "bloom_op_w4_read": (I32, [P, P, C.c_int64, P]),
    "bloom_op_linear_w4": (I32, [P, P, C.c_int64, I32, P, I32, P, C.c_int64, I32, P, C.c_size_t, P, P]),
    "bloom_op_linear_w4_workspace": (C.c_size_t, [P, I32]),
    "bloom_op_linear_w4_wait_ns": (I32, [I32]),
    "bloom_op_lmhead_argmax_noalloc": (I32, [P, P, I32, I32, I32, P, P, P]),
}
EXPORTS = tuple(_SIGS)


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def check(status: int):
    if status != BLOOM_OK:
        raise BloomError(status, lib().bloom_last_error().decode())


def _p(t: Optional[torch.Tensor]):
    return None if t is None else P(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return P(s.cuda_stream)


class KV:
    """A caller-owned KV cache (one device byte buffer) and its descriptor;
    with offload_from < n_layer the K and V of layers [offload_from, n_layer)
    live in a second, page-locked host buffer the kernels read directly."""

    def __init__(self, model: "Model", batch: int, max_seq: int, stream=None,
                 offload_from: Optional[int] = None):
        self.offload_from = model.n_layer if offload_from is None else int(offload_from)
        self.host = None
        if self.offload_from >= model.n_layer:
            n = lib().bloom_kv_bytes(C.byref(model.cfg), batch, max_seq)
            if n == 0:
                raise BloomError(1, "bloom_kv_bytes rejected the arguments")
            hn = 0
        else:
            dn, hb = C.c_size_t(), C.c_size_t()
            check(lib().bloom_kv_bytes_offload(C.byref(model.cfg), batch, max_seq,
                                               self.offload_from, C.byref(dn), C.byref(hb)))
            n, hn = dn.value, hb.value
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=model.device)
        off = (-self.buf.data_ptr()) % 256
        self.view = self.buf[off:off + n]
        self.c = KVC()
        if hn == 0:
            check(lib().bloom_kv_init(model.h, C.byref(self.c), P(self.view.data_ptr()), n, batch,
                                      max_seq, _stream(stream)))
        else:
            self.host = torch.empty(hn + 256, dtype=torch.uint8, pin_memory=True)
            hoff = (-self.host.data_ptr()) % 256
            self.host_view = self.host[hoff:hoff + hn]
            check(lib().bloom_kv_init_offload(model.h, C.byref(self.c), P(self.view.data_ptr()), n,
                                              P(self.host_view.data_ptr()), hn, batch, max_seq,
                                              self.offload_from, _stream(stream)))

    @property
    def len(self) -> int:
        return self.c.len

    @property
    def batch(self) -> int:
        return self.c.batch

    def row_len(self, b: int) -> int:
        return self.c.row_len[b]

    def row_active(self, b: int) -> bool:
        return bool(self.c.row_active[b])

    def tensors(self, model: "Model"):
        """Views of the cache regions (len, active, next_pos, pos, K, V) for inspection."""
        sh = model.shape
        B, S = self.c.batch, self.c.max_seq
        al = lambda x: (x + 255) // 256 * 256
        off_len = 256
        off_act = al(off_len + 4 * B)
        off_np = al(off_act + 4 * B)
        off_pos = al(off_np + 4 * B)
        layer = B * sh.n_head * S * sh.head_dim * 2
        nd = min(self.offload_from, model.n_layer)   # layers in the device buffer
        off_k = al(off_pos + 4 * B * S)
        off_v = al(off_k + layer * nd)
        v = self.view
        i32 = lambda a, n: v[a:a + 4 * n].view(torch.int32)
        bf = lambda buf, a, nl: buf[a:a + layer * nl].view(torch.bfloat16).view(
            nl, B, sh.n_head, S, sh.head_dim)
        out = {"len": i32(off_len, B), "active": i32(off_act, B), "next_pos": i32(off_np, B),
               "pos": i32(off_pos, B * S).view(B, S), "k": bf(v, off_k, nd), "v": bf(v, off_v, nd)}
        if self.host is not None:
            nh = model.n_layer - nd
            out["k_host"] = bf(self.host_view, 0, nh)
            out["v_host"] = bf(self.host_view, al(layer * nh), nh)
        return out


class Model:
    """A BLOOM stack on the current CUDA device, weights borrowed from torch tensors."""

    def __init__(self, weights: synth.Weights, max_batch: int, max_tokens: int, max_seq: int,
                 flags: int = 0, n_layer: Optional[int] = None, wait_us: int = 0):
        sh = weights.shape
        self.shape = sh
        self.weights = weights
        self.n_layer = len(weights.layers) if n_layer is None else n_layer
        self.device = weights.word_emb.device
        self.cfg = Config(self.n_layer, sh.hidden, sh.n_head, sh.ffn, sh.vocab, sh.ln_eps,
                          1 if sh.int8 else 0, max_batch, max_tokens, max_seq, flags, wait_us)
        arr = (LayerWeights * self.n_layer)()
        for i in range(self.n_layer):
            L = weights.layers[i]

            def lin(name):
                if sh.int8:
                    return Linear(_p(L["q_" + name]), _p(L["s_" + name]), _p(L["b_" + name]))
                return Linear(_p(L["w_" + name]), None, _p(L["b_" + name]))

            arr[i] = LayerWeights(_p(L["ln1_g"]), _p(L["ln1_b"]), lin("qkv"), lin("o"),
                                  _p(L["ln2_g"]), _p(L["ln2_b"]), lin("up"), lin("down"))
        self._arr = arr
        self._wc = WeightsC(_p(weights.word_emb), _p(weights.emb_ln_g), _p(weights.emb_ln_b),
                            _p(weights.lnf_g), _p(weights.lnf_b),
                            C.cast(arr, C.POINTER(LayerWeights)))
        h = P()
        check(lib().bloom_create(C.byref(self.cfg), C.byref(self._wc), C.byref(h)))
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().bloom_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def decode_launches(self, batch: int) -> int:
        return lib().bloom_decode_launches(self.h, batch)

    def new_kv(self, batch: int, max_seq: int, stream=None, offload_from: Optional[int] = None) -> KV:
        return KV(self, batch, max_seq, stream, offload_from)

    def prefill(self, kv: KV, tokens, mask, out_tokens=None, logits=None, stream=None):
        B, T = tokens.shape
        if out_tokens is None:
            out_tokens = torch.empty(B, dtype=torch.int32, device=self.device)
        check(lib().bloom_prefill(self.h, C.byref(kv.c), _p(tokens), _p(mask), B, T,
                                  _p(out_tokens), _p(logits), _stream(stream)))
        return out_tokens

    def decode_step(self, kv: KV, next_tokens, out_tokens=None, logits=None, stream=None):
        if out_tokens is None:
            out_tokens = torch.empty(kv.batch, dtype=torch.int32, device=self.device)
        check(lib().bloom_decode_step(self.h, C.byref(kv.c), _p(next_tokens), _p(out_tokens),
                                      _p(logits), _stream(stream)))
        return out_tokens

    def decode_step_sampled(self, kv: KV, next_tokens, temperature, top_p, u, logits,
                            out_tokens=None, stream=None):
        """One decode step, then each active row's token sampled with its own
        temperature / top-p at the caller's uniform u (device float32 [B] each;
        logits: device float32 [B][V] scratch, written)."""
        if out_tokens is None:
            out_tokens = torch.empty(kv.batch, dtype=torch.int32, device=self.device)
        check(lib().bloom_decode_step_sampled(self.h, C.byref(kv.c), _p(next_tokens),
                                              _p(out_tokens), _p(logits), _p(temperature),
                                              _p(top_p), _p(u), _stream(stream)))
        return out_tokens

    def kv_admit(self, kv: KV, rows, tokens, mask, out_tokens=None, logits=None, stream=None):
        """Prefill new prompts (device tokens / mask [n][T]) into cache rows `rows`."""
        n, T = tokens.shape
        r = (C.c_int32 * n)(*[int(v) for v in rows])
        if out_tokens is None:
            out_tokens = torch.empty(n, dtype=torch.int32, device=self.device)
        check(lib().bloom_kv_admit(self.h, C.byref(kv.c), r, n, _p(tokens), _p(mask), T,
                                   _p(out_tokens), _p(logits), _stream(stream)))
        return out_tokens

    def kv_retire(self, kv: KV, rows, stream=None):
        """Rows `rows` leave the batch (decode steps skip them)."""
        r = (C.c_int32 * len(rows))(*[int(v) for v in rows])
        check(lib().bloom_kv_retire(self.h, C.byref(kv.c), r, len(rows), _stream(stream)))

    def generate(self, kv: KV, tokens_host, mask_host, n_new: int, out_host=None, stream=None):
        """Greedy generation from host buffers; returns host int32 [n_new, B]."""
        B, T = tokens_host.shape
        if out_host is None:
            out_host = torch.empty(n_new, B, dtype=torch.int32)
        check(lib().bloom_generate(self.h, C.byref(kv.c), _p(tokens_host), _p(mask_host), B, T,
                                   n_new, _p(out_host), _stream(stream)))
        return out_host

    def decode_profile(self, kv: KV, next_tokens, out_tokens=None, cap: int = 4096, stream=None):
        """One decode step launched kernel by kernel with an event after each;
        returns [(op, kernel, ms)] in launch order (names in OPS / KERNELS)."""
        if out_tokens is None:
            out_tokens = torch.empty(kv.batch, dtype=torch.int32, device=self.device)
        codes = (C.c_int32 * cap)()
        ms = (C.c_float * cap)()
        n = C.c_int32(0)
        check(lib().bloom_decode_profile(self.h, C.byref(kv.c), _p(next_tokens), _p(out_tokens),
                                         codes, ms, cap, C.byref(n), _stream(stream)))
        return [(OPS[codes[i] & 0xff], KERNELS[codes[i] >> 8], float(ms[i]))
                for i in range(n.value)]

    def check_device(self, stream=None):
        check(lib().bloom_check_device(self.h, _stream(stream)))

    def layer_decode(self, kv: KV, layer: int, x, stream=None):
        check(lib().bloom_layer_decode(self.h, C.byref(kv.c), layer, _p(x), _stream(stream)))

    def kv_set_prompt(self, kv: KV, mask, stream=None):
        B, T = mask.shape
        check(lib().bloom_kv_set_prompt(self.h, C.byref(kv.c), _p(mask), B, T, _stream(stream)))

    def layer_prefill(self, kv: KV, layer: int, x, B: int, T: int, stream=None):
        check(lib().bloom_layer_prefill(self.h, C.byref(kv.c), layer, _p(x), B, T,
                                        _stream(stream)))

    def head(self, x, out_tokens=None, logits=None, stream=None):
        B = x.shape[0]
        if out_tokens is None:
            out_tokens = torch.empty(B, dtype=torch.int32, device=self.device)
        check(lib().bloom_head(self.h, _p(x), B, _p(out_tokens), _p(logits), _stream(stream)))
        return out_tokens

    def lm_head(self, xn, out_tokens, logits=None, stream=None):
        """The tied head + argmax kernel alone on normalised rows xn [B, h]."""
        check(lib().bloom_lm_head(self.h, _p(xn), xn.shape[0], _p(out_tokens), _p(logits),
                                  _stream(stream)))
        return out_tokens

    def embed(self, tokens, x=None, stream=None):
        n = tokens.numel()
        if x is None:
            x = torch.empty(n, self.shape.hidden, dtype=torch.float32, device=self.device)
        check(lib().bloom_embed(self.h, _p(tokens), n, _p(x), _stream(stream)))
        return x


# ----------------------------------------------------------------- operators
def op_layernorm(x, g=None, b=None, eps=1e-5, y=None, stream=None):
    rows, h = x.shape
    if y is None:
        y = torch.empty_like(x)
    check(lib().bloom_op_layernorm(_p(x), _p(g), _p(b), rows, h, eps, _p(y), _stream(stream)))
    return y


def op_linear(x, w=None, bias=None, q=None, scale=None, epilogue=EPI_STORE, y=None,
              stream=None):
    M, K = x.shape
    N = (w if w is not None else q).shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    lin = Linear(_p(w if w is not None else q), _p(scale), _p(bias))
    check(lib().bloom_op_linear(C.byref(lin), 0 if w is not None else 1, _p(x), M, N, K,
                                epilogue, _p(y), _stream(stream)))
    return y


def op_gemm(x, w, bias=None, epilogue=EPI_STORE, y=None, stream=None):
    """bf16 linear layer on the tensor-core (tcgen05) GEMM used by prefill."""
    M, K = x.shape
    N = w.shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    lin = Linear(_p(w), None, _p(bias))
    check(lib().bloom_op_gemm(C.byref(lin), _p(x), M, N, K, epilogue, _p(y), _stream(stream)))
    return y


def op_linear_tc(x, w=None, bias=None, q=None, scale=None, epilogue=EPI_STORE, y=None,
                 stream=None):
    """Linear layer on the tensor-core decode kernel: bf16 weights w (M <= 256
    tokens) or int8 codes q with bf16 row scales (M <= 128)."""
    M, K = x.shape
    N = (w if w is not None else q).shape[0]
    if y is None:
        y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    lin = Linear(_p(w if w is not None else q), _p(scale), _p(bias))
    check(lib().bloom_op_linear_tc(C.byref(lin), 0 if w is not None else 1, _p(x), M, N, K,
                                   epilogue, _p(y), _stream(stream)))
    return y


def op_attn_decode(q, k_cache, v_cache, pos, slopes, length: int, splits: int = 0, o=None,
                   stream=None):
    B, n, S, d = k_cache.shape
    if o is None:
        o = torch.empty(B, n * d, dtype=torch.bfloat16, device=q.device)
    check(lib().bloom_op_attn_decode(_p(q), _p(k_cache), _p(v_cache), _p(pos), _p(slopes), B, n,
                                     d, S, length, splits, _p(o), _stream(stream)))
    return o


def op_lmhead_argmax(x, emb, logits: bool = True, stream=None):
    M, K = x.shape
    V = emb.shape[0]
    tok = torch.empty(M, dtype=torch.int32, device=x.device)
    lg = torch.empty(M, V, dtype=torch.float32, device=x.device) if logits else None
    check(lib().bloom_op_lmhead_argmax(_p(x), _p(emb), M, V, K, _p(tok), _p(lg),
                                       _stream(stream)))
    return tok, lg


def op_sample(logits, temperature, top_p, u, out=None, stream=None):
    """Temperature + top-p sampling of float32 logits [B][V] (rows may be
    strided) with per-row device float32 [B] temperature, top_p, u."""
    B, V = logits.shape
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    check(lib().bloom_op_sample(_p(logits), B, V, logits.stride(0), _p(temperature), _p(top_p),
                                _p(u), _p(out), _stream(stream)))
    return out


def op_lmhead_argmax_noalloc(x, emb, logits: bool = True, stream=None):
    """bloom_op_lmhead_argmax without allocation (fixed in-library scratch)."""
    M, K = x.shape
    V = emb.shape[0]
    tok = torch.empty(M, dtype=torch.int32, device=x.device)
    lg = torch.empty(M, V, dtype=torch.float32, device=x.device) if logits else None
    check(lib().bloom_op_lmhead_argmax_noalloc(_p(x), _p(emb), M, V, K, _p(tok), _p(lg),
                                               _stream(stream)))
    return tok, lg


def _bad(msg: str):
    raise BloomError(1, msg)


def _expected(name, t, dtype, shape, device, what="contiguous"):
    _bad(f"{name}: {what} {dtype} {tuple(shape)} on {device} expected, "
         f"got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _dev(name: str, t, dtype, shape, device):
    """A contiguous device tensor of that type and shape, or an error; its address
    (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _expected(name, t, dtype, shape, device)
    return t.data_ptr()


def _elsewhere(device, stream):
    """None where a call on `stream` (None: the device's current one) runs on what is
    current already; else a context that makes its device and stream current, so that
    what is allocated inside belongs to that stream."""
    if device.type != "cuda":
        _bad(f"tensors on a CUDA device expected, got {device}")
    if stream is None:
        if device.index == torch.cuda.current_device():
            return None
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        _bad(f"stream on {stream.device}, tensors on {device}")
    return torch.cuda.stream(stream)


def _raw_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


KV8_BLOCK = 32
_KV8_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class KV8(NamedTuple):
    """An 8-bit KV cache of one layer: value = code * scale.

    k, v: codes, int8 or float8_e4m3fn [B][n_kv][S][d], d 64 or 128; k_scale,
    v_scale: float32 [B][n_kv][ceil(S / 32)], one for every 32 slots of a head."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, batch: int, n_kv: int, max_seq: int, d: int, codes=torch.int8, device="cuda"):
        """A cache of zeros; codes torch.int8 or torch.float8_e4m3fn."""
        kv = [torch.zeros(batch, n_kv, max_seq, d, dtype=codes, device=device) for _ in range(2)]
        sc = [torch.zeros(batch, n_kv, -(-max_seq // KV8_BLOCK), device=device) for _ in range(2)]
        return cls(*kv, *sc)

    def c(self) -> KV8C:
        """The C descriptor (bloom_kv8), after checking types, shapes and devices."""
        k, v, ks, vs = self
        dt, shape, dev = k.dtype, k.shape, k.device
        codes = _KV8_CODES.get(dt)
        if codes is None or len(shape) != 4 or not k.is_contiguous():
            _bad(f"cache codes: contiguous int8 or float8_e4m3fn [B][n][S][d] expected, got "
                 f"{dt} {tuple(shape)}, strides {k.stride()}")
        B, n, S, d = shape
        sc = (B, n, -(-S // KV8_BLOCK))
        return KV8C(k.data_ptr(), _dev("v", v, dt, shape, dev), _dev("k_scale", ks, _F32, sc, dev),
                    _dev("v_scale", vs, _F32, sc, dev), codes, B, n, S, d)


def _kv8_values(name: str, t, shape, device):
    """(address, strides) of a bf16 [B][T][n][d] view whose d elements lie together."""
    st = t.stride()
    if t.dtype is not _BF16 or t.shape != shape or t.device != device or st[3] != 1:
        _expected(name, t, _BF16, shape, device, "unit last stride,")
    B, T, n, _ = shape      # the stride of a dimension of one element means nothing
    return t.data_ptr(), _I64x3(st[0] if B > 1 else 0, st[1] if T > 1 else 0, st[2] if n > 1 else 0)


_I64x3 = C.c_int64 * 3


def op_kv8_write(kv: KV8, k, v, start, count=None, mask=None, flag=None, stream=None):
    """Quantise new keys and values k, v (bf16 [B][T][n][d], any strides that are
    multiples of 8) into slots start[b] + t of the cache, in place: start int32
    [B], -1 for an idle row; count int32 [B], tokens of each row (None: T); mask
    uint8 [B][T], 0 for pad slots; flag int32 [1] that errors are recorded in."""
    c, dev = kv.c(), kv.k.device
    if k.dim() != 4:
        _bad(f"k: [B][T][n][d] expected, got {tuple(k.shape)}")
    B, T = c.batch, k.shape[1]
    shape = (B, T, c.n_kv, c.d)
    kp, ks = _kv8_values("k", k, shape, dev)
    vp, vs = _kv8_values("v", v, shape, dev)
    sp, cp = _dev("start", start, _I32, (B,), dev), _dev("count", count, _I32, (B,), dev)
    mp, fp = _dev("mask", mask, _U8, (B, T), dev), _dev("flag", flag, _I32, (1,), dev)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_kv8_write(kv, k, v, start, count, mask, flag)
    st = lib().bloom_op_kv8_write(C.byref(c), kp, ks, vp, vs, T, sp, cp, mp, fp, _raw_stream(dev))
    if st:
        check(st)


def op_kv8_read(kv: KV8, start, T: int, count=None, k=None, v=None, flag=None, stream=None):
    """Slots start[b] + t, t < T, of the cache as bf16 (k, v) [B][T][n][d]: views
    given, or new tensors.  Zeros for idle rows (start -1), for t >= count[b]
    and beyond the cache."""
    c, dev = kv.c(), kv.k.device
    if T < 0:
        _bad(f"T={T}")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_kv8_read(kv, start, T, count, k, v, flag)
    B, n, d = c.batch, c.n_kv, c.d
    shape = (B, T, n, d)
    ks = vs = None
    if k is None or v is None:
        dense = _I64x3(T * n * d, n * d, d)
    if k is None:
        k, ks = torch.empty(shape, dtype=_BF16, device=dev), dense
        kp = k.data_ptr()
    if v is None:
        v, vs = torch.empty(shape, dtype=_BF16, device=dev), dense
        vp = v.data_ptr()
    if ks is None:
        kp, ks = _kv8_values("k", k, shape, dev)
    if vs is None:
        vp, vs = _kv8_values("v", v, shape, dev)
    st = lib().bloom_op_kv8_read(
        C.byref(c), kp, ks, vp, vs, T, _dev("start", start, _I32, (B,), dev),
        _dev("count", count, _I32, (B,), dev), _dev("flag", flag, _I32, (1,), dev),
        _raw_stream(dev))
    if st:
        check(st)
    return k, v


def op_attn_decode_kv8(q, kv: KV8, pos, slopes, lens, o=None, workspace=None, flag=None,
                       stream=None):
    """Decode attention over an 8-bit cache: q bf16 [B][T][n][d] for the last T
    tokens of every row (or [B][n][d], T = 1), whose keys are in the cache; pos
    int32 [B][S], -1 masked; slopes float32 [n] or None; lens int32 [B], slots
    filled.  Returns o bf16 [B][T][n * d] (or [B][n * d]).  workspace: uint8,
    bloom_op_attn_decode_kv8_workspace() bytes, None to allocate it."""
    c, dev = kv.c(), kv.k.device
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_attn_decode_kv8(q, kv, pos, slopes, lens, o, workspace, flag)
    B, d = c.batch, c.d
    if q.dim() == 4:
        T, n = q.shape[1:3]
        qp, oshape = _dev("q", q, _BF16, (B, T, n, d), dev), (B, T, n * d)
    elif q.dim() == 3:
        T, n = 1, q.shape[1]
        qp, oshape = _dev("q", q, _BF16, (B, n, d), dev), (B, n * d)
    else:
        _bad(f"q: [B][T][n][d] or [B][n][d] expected, got {tuple(q.shape)}")
    pp, sp = _dev("pos", pos, _I32, (B, c.max_seq), dev), _dev("slopes", slopes, _F32, (n,), dev)
    lp, fp = _dev("lens", lens, _I32, (B,), dev), _dev("flag", flag, _I32, (1,), dev)
    L, cr = lib(), C.byref(c)
    if o is None:
        o = torch.empty(oshape, dtype=_BF16, device=dev)
    wp, wn = None, 0
    if workspace is not None:
        if workspace.dtype is not _U8 or workspace.dim() != 1:
            _bad(f"workspace: uint8 [bytes] expected, got {workspace.dtype} {tuple(workspace.shape)}")
        wn = workspace.numel()
        wp = _dev("workspace", workspace, _U8, (wn,), dev)
    else:
        wn = L.bloom_op_attn_decode_kv8_workspace(cr, T, n)
        if wn:
            workspace = torch.empty(wn, dtype=_U8, device=dev)
            wp = workspace.data_ptr()
    st = L.bloom_op_attn_decode_kv8(cr, qp, pp, sp, lp, T, n, _dev("o", o, _BF16, oshape, dev), wp,
                                    wn, fp, _raw_stream(dev))
    if st:
        check(st)
    return o


def op_sample_filtered(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None,
                       stream=None):
    """Tokens of float32 logits [B][V] (rows may be strided) drawn at uniform numbers u
    (float32 [B], or [B][J] for J draws a row) with per-row temperature, top_p, min_p
    (float32 [B]) and top_k (int32 [B]), None for none: int32, shaped like u."""
    dev = logits.device
    if logits.dtype is not _F32 or logits.dim() != 2 or logits.stride(1) != 1:
        _bad(f"logits: float32 [B][V] with unit last stride expected, got {logits.dtype} "
             f"{tuple(logits.shape)}, strides {logits.stride()}")
    B, V = logits.shape
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_sample_filtered(logits, u, temperature, top_k, top_p, min_p, out)
    J = u.shape[1] if u.dim() == 2 else 1
    shape = (B, J) if u.dim() == 2 else (B,)
    if max(B, V, J) >= 2 ** 31:         # would wrap in the call
        _bad(f"logits {(B, V)}, {J} draws: sizes below 2^31 expected")
    up, row = _dev("u", u, _F32, shape, dev), (B,)
    if out is None:
        out = torch.empty(shape, dtype=_I32, device=dev)
        op = out.data_ptr()
    else:
        op = _dev("out", out, _I32, shape, dev)
    st = lib().bloom_op_sample_filtered(
        logits.data_ptr(), B, V, logits.stride(0) if B > 1 else V,
        _dev("temperature", temperature, _F32, row, dev), _dev("top_k", top_k, _I32, row, dev),
        _dev("top_p", top_p, _F32, row, dev), _dev("min_p", min_p, _F32, row, dev), up, J, op,
        _raw_stream(dev))
    if st:
        check(st)
    return out


def op_logprobs(logits, tokens=None, top: int = 0, stream=None):
    """Log probabilities of tokens (int32 [B][J] or [B]; -1: none) under softmax of
    float32 logits [B][V] (rows may be strided), the rows' entropies, and their
    `top` <= 32 most probable tokens: (logp like tokens or None, entropy [B],
    top_ids int32 [B][top], top_logp [B][top])."""
    dev = logits.device
    if logits.dtype is not _F32 or logits.dim() != 2 or logits.stride(1) != 1:
        _bad(f"logits: float32 [B][V] with unit last stride expected, got {logits.dtype} "
             f"{tuple(logits.shape)}, strides {logits.stride()}")
    B, V = logits.shape
    if not 0 <= top <= 32:
        _bad(f"top={top}: 0 to 32 expected")
    J, tp, logp, lp = 0, None, None, None
    if tokens is not None:
        J = tokens.shape[1] if tokens.dim() == 2 else 1
        tp = _dev("tokens", tokens, _I32, (B, J) if tokens.dim() == 2 else (B,), dev)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_logprobs(logits, tokens, top)
    if tokens is not None:
        logp = torch.empty(tokens.shape, device=dev)
        lp = logp.data_ptr()
    entropy = torch.empty(B, device=dev)
    ids = torch.empty((B, top), dtype=_I32, device=dev)
    lps = torch.empty((B, top), device=dev)
    st = lib().bloom_op_logprobs(logits.data_ptr(), B, V, logits.stride(0) if B > 1 else V, tp, J,
                                 lp, entropy.data_ptr(), top, ids.data_ptr(), lps.data_ptr(),
                                 _raw_stream(dev))
    if st:
        check(st)
    return logp, entropy, ids, lps


def _w4_bytes(n: int, k: int, group: int) -> int:
    # sizes past 32 bits would wrap in the call
    size = lib().bloom_w4_bytes(n, k, group) if max(n, k, group) < 2 ** 31 else 0
    if size == 0:
        _bad(f"n={n}, k={k}, group={group}: k a multiple of 8, groups of 32, 64 or 128 expected")
    return size


class W4:
    """4-bit weights [n][k] with group scales: value = code * scale, codes -7 .. 7, a
    bf16 scale for every `group` (32, 64 or 128) neighbouring weights of a row.  tiles:
    uint8 [bloom_w4_bytes(n, k, group)], in the order that the linear layer reads them."""
    __slots__ = ("tiles", "n", "k", "group", "device", "ref", "_c")

    def __init__(self, tiles: torch.Tensor, n: int, k: int, group: int):
        size = _w4_bytes(n, k, group)
        self._c = W4C(_dev("tiles", tiles, _U8, (size,), tiles.device), n, k, group)
        self.ref = C.byref(self._c)         # the C descriptor (bloom_w4)
        self.tiles, self.n, self.k, self.group, self.device = tiles, n, k, group, tiles.device

    @classmethod
    def empty(cls, n: int, k: int, group: int = 64, device="cuda"):
        """Room for [n][k] weights (k a multiple of 8), not initialised."""
        return cls(torch.empty(_w4_bytes(n, k, group), dtype=_U8, device=device), n, k, group)


def _rows(name: str, t, dtype, shape, device):
    """(address, row stride) of a [rows][columns] tensor whose columns lie together."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or t.stride(1) != 1:
        _expected(name, t, dtype, shape, device, "unit last stride,")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]   # one row: its stride means nothing


def op_w4_quantize(w, group: Optional[int] = None, out: Optional[W4] = None, stream=None) -> W4:
    """bf16 weights w [n][k] (rows may be strided, k a multiple of 8) in 4 bits: into
    `out`, in its groups, or new tiles in groups of `group` (64 unless given)."""
    dev = w.device
    if w.dim() != 2:
        _bad(f"w: [n][k] expected, got {tuple(w.shape)}")
    n, k = w.shape
    if out is not None and (out.n, out.k, out.device) != (n, k, dev):
        _bad(f"out: weights {(n, k)} on {dev} expected, got {(out.n, out.k)} on {out.device}")
    if out is not None and group is not None and group != out.group:
        _bad(f"group={group}: out has groups of {out.group}")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_w4_quantize(w, group, out)
    wp, ld = _rows("w", w, _BF16, (n, k), dev)
    if out is None:
        out = W4.empty(n, k, 64 if group is None else group, dev)
    st = lib().bloom_op_w4_quantize(wp, ld, out.ref, _raw_stream(dev))
    if st:
        check(st)
    return out


def op_w4_read(w4: W4, out=None, stream=None):
    """The weights back as bf16 [n][k] (rows of `out` may be strided): for prompts, which
    run on op_gemm, or to look at what the codes stand for."""
    dev = w4.device
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_w4_read(w4, out)
    n, k = w4.n, w4.k
    if out is None:
        out = torch.empty((n, k), dtype=_BF16, device=dev)
    wp, ld = _rows("out", out, _BF16, (n, k), dev)
    st = lib().bloom_op_w4_read(w4.ref, wp, ld, _raw_stream(dev))
    if st:
        check(st)
    return out


def op_linear_w4(x, w4: W4, bias=None, epilogue=EPI_STORE, y=None, dtype=torch.bfloat16, workspace=None,
                 flag=None, stream=None):
    """Linear layer of a decode step over 4-bit weights: x bf16 [M][k], bias bf16 [n];
    y bf16 or float32 [M][n], given (required for EPI_RESID, which adds to it) or new, of
    `dtype`.  Rows of x and y may be strided.  workspace: uint8, bloom_op_linear_w4_workspace()
    bytes, None to allocate it.  flag int32 [1] that errors are recorded in."""
    dev = x.device
    if x.dim() != 2:
        _bad(f"x: [M][k] expected, got {tuple(x.shape)}")
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return op_linear_w4(x, w4, bias, epilogue, y, dtype, workspace, flag)
    if w4.device != dev:
        _bad(f"weights on {w4.device}, x on {dev}")
    M, n = x.shape[0], w4.n
    xp, ldx = _rows("x", x, _BF16, (M, w4.k), dev)
    if M > 1 << 20:
        _bad(f"M={M}: at most {1 << 20} tokens")
    if y is None:
        if epilogue == EPI_RESID:
            _bad("y: EPI_RESID adds to it")
        if dtype is not _BF16 and dtype is not _F32:
            _bad(f"dtype={dtype}: bfloat16 or float32 expected")
        f32 = dtype is _F32
        y = torch.empty((M, n), dtype=dtype, device=dev)
        yp, ldy = y.data_ptr(), n
    else:
        f32 = y.dtype is _F32
        yp, ldy = _rows("y", y, _F32 if f32 else _BF16, (M, n), dev)
    bp = None if bias is None else _dev("bias", bias, _BF16, (n,), dev)
    fp = None if flag is None else _dev("flag", flag, _I32, (1,), dev)
    L = lib()
    wp, wn = None, 0
    if workspace is not None:
        if workspace.dtype is not _U8 or workspace.dim() != 1:
            _bad(f"workspace: uint8 [bytes] expected, got {workspace.dtype} {tuple(workspace.shape)}")
        wn = workspace.numel()
        wp = _dev("workspace", workspace, _U8, (wn,), dev)
    elif M > 8:
        wn = L.bloom_op_linear_w4_workspace(w4.ref, M)
        workspace = torch.empty(wn, dtype=_U8, device=dev)
        wp = workspace.data_ptr()
    st = L.bloom_op_linear_w4(w4.ref, xp, ldx, M, bp, epilogue, yp, ldy, f32, wp, wn, fp, _raw_stream(dev))
    if st:
        check(st)
    return y
