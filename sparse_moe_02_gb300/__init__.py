"""Python binding of libmoe, the GB300 (sm_103a) mixture-of-experts FFN layer.

Argument marshalling only: every function here forwards to the C entry point of the same
name declared in include/moe.h and returns its status code; all arithmetic runs in the CUDA
kernels of libmoe.so.  There is no fallback: if the library is missing or cannot be loaded,
import-time use fails loudly.

MoeLayer is a small convenience wrapper that takes torch CUDA tensors (PyTorch is used only
for device memory and streams) and raises MoeError on a non-zero status.  PagedAttention is the
same for the attention step over a paged 4-bit cache (include/attn.h).

With MOE_DEBUG_LIBRARY=1 in the environment the binding loads libmoe_debug.so instead: the same
library built with MOE_DEBUG, which checks every routing it produces (moe_check_routing) and
records a failure in the handle's device error word.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_debug.so" if os.environ.get("MOE_DEBUG_LIBRARY") == "1"
                        else "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_ALIGNMENT = 3
MOE_ERR_CUDA = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_DEVICE = 6
MOE_ERR_NO_MEMORY = 7

MOE_SCHEDULE_AUTO = 0
MOE_SCHEDULE_GEMM = 1
MOE_SCHEDULE_GEMV = 2

EXPORTS = ("moe_create", "moe_route", "moe_forward", "moe_forward_host", "moe_get_device_error",
           "moe_destroy", "moe_status_string", "moe_last_cuda_error", "moe_profile_begin",
           "moe_profile_end", "moe_route_one_noalloc", "moe_create_q4", "moe_read_probe",
           "moe_test_expire_waits", "gdn_scan", "moe_check_routing")

ATTN_EXPORTS = ("attn_create", "attn_destroy", "attn_get_device_error", "attn_plan",
                "attn_qk_norm_rope", "attn_kv4_append", "attn_kv4_read", "attn_kv4_forward")

# kernel order reported by moe_profile_end
KERNELS_GEMM = ("router_topk", "route_plan_scatter", "experts", "combine")
KERNELS_GEMV = ("decode_router_shared", "decode_gateup", "decode_down_combine")

_c_int, _c_void_p = ctypes.c_int, ctypes.c_void_p


class moe_config(ctypes.Structure):
    _fields_ = [("d", _c_int), ("n_experts", _c_int), ("top_k", _c_int), ("ffn_dim", _c_int),
                ("shared_ffn_dim", _c_int), ("max_tokens", _c_int), ("schedule", _c_int),
                ("chunk_tokens", _c_int)]


class moe_weights(ctypes.Structure):
    _fields_ = [("w_router", _c_void_p), ("router_bias", _c_void_p), ("w_gate", _c_void_p),
                ("w_up", _c_void_p), ("w_down", _c_void_p), ("ws_gate", _c_void_p),
                ("ws_up", _c_void_p), ("ws_down", _c_void_p)]


class moe_q4_matrix(ctypes.Structure):
    _fields_ = [("codes", _c_void_p), ("scales", _c_void_p), ("biases", _c_void_p)]


class moe_weights_q4(ctypes.Structure):
    _fields_ = [("w_router", _c_void_p), ("router_bias", _c_void_p),
                ("w_gate", moe_q4_matrix), ("w_up", moe_q4_matrix), ("w_down", moe_q4_matrix),
                ("ws_gate", moe_q4_matrix), ("ws_up", moe_q4_matrix),
                ("ws_down", moe_q4_matrix)]


class attn_config(ctypes.Structure):
    _fields_ = [("n_q_heads", _c_int), ("n_kv_heads", _c_int), ("head_dim", _c_int),
                ("page_size", _c_int), ("n_pages", _c_int), ("max_requests", _c_int),
                ("scale", ctypes.c_float)]


_lib = None


def lib():
    """The loaded libmoe.so (raises OSError if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{os.path.basename(LIB_PATH)} not built ({LIB_PATH}); "
                          "run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_create.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights),
                                 ctypes.POINTER(_c_void_p)]
        L.moe_read_probe.argtypes = [_c_void_p, ctypes.c_size_t, _c_void_p, _c_void_p]
        L.moe_create_q4.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(moe_weights_q4),
                                    ctypes.POINTER(_c_void_p)]
        L.moe_route.argtypes = [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                _c_void_p, _c_void_p]
        L.moe_forward.argtypes = [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p]
        L.moe_forward_host.argtypes = [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p]
        L.moe_get_device_error.argtypes = [_c_void_p, _c_void_p]
        L.moe_destroy.argtypes = [_c_void_p]
        L.moe_status_string.argtypes = [_c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_cuda_error.argtypes = []
        L.moe_profile_begin.argtypes = [_c_void_p, _c_int]
        L.moe_profile_end.argtypes = [_c_void_p, ctypes.POINTER(ctypes.c_float), _c_int,
                                      ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]
        L.moe_route_one_noalloc.argtypes = [_c_void_p, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                            _c_void_p, _c_void_p]
        L.moe_test_expire_waits.argtypes = [_c_void_p, _c_int]
        L.moe_check_routing.argtypes = [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p,
                                        _c_void_p]
        L.gdn_scan.argtypes = [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                               _c_void_p, _c_void_p, ctypes.c_int64, _c_int, _c_int, _c_int,
                               _c_void_p]
        i64 = ctypes.c_int64
        L.attn_create.argtypes = [ctypes.POINTER(attn_config), ctypes.POINTER(_c_void_p)]
        L.attn_destroy.argtypes = [_c_void_p]
        L.attn_get_device_error.argtypes = [_c_void_p, _c_void_p]
        L.attn_plan.argtypes = [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p, _c_int,
                                _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p, _c_void_p,
                                _c_void_p, _c_void_p, _c_void_p, _c_void_p]
        L.attn_qk_norm_rope.argtypes = [_c_void_p, _c_void_p, i64, _c_void_p, i64, _c_void_p,
                                        _c_void_p, _c_void_p, ctypes.c_float, _c_void_p, _c_int,
                                        _c_int, _c_int, _c_int, _c_void_p, i64, _c_void_p, i64,
                                        _c_void_p]
        L.attn_kv4_append.argtypes = [_c_void_p, _c_void_p, i64, _c_void_p, i64, _c_void_p,
                                      _c_int, _c_void_p, _c_void_p]
        L.attn_kv4_read.argtypes = [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, i64,
                                    _c_void_p, i64, _c_void_p]
        L.attn_kv4_forward.argtypes = [_c_void_p, _c_void_p, i64, _c_void_p, _c_void_p, _c_int,
                                       _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                       _c_void_p, i64, _c_void_p]
        for fn in ATTN_EXPORTS:
            getattr(L, fn).restype = _c_int
        for fn in ("moe_create", "moe_create_q4", "moe_read_probe", "moe_route", "moe_forward", "moe_forward_host",
                   "moe_get_device_error", "moe_destroy", "moe_last_cuda_error",
                   "moe_profile_begin", "moe_profile_end", "moe_route_one_noalloc",
                   "moe_test_expire_waits", "gdn_scan", "moe_check_routing"):
            getattr(L, fn).restype = _c_int
        _lib = L
    return _lib


def moe_create(cfg, weights):
    """Returns (status, handle)."""
    h = _c_void_p()
    st = lib().moe_create(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(h))
    return st, h


def moe_create_q4(cfg, weights_q4):
    """Returns (status, handle) for 4-bit experts (moe_weights_q4)."""
    h = _c_void_p()
    st = lib().moe_create_q4(ctypes.byref(cfg), ctypes.byref(weights_q4), ctypes.byref(h))
    return st, h


def moe_read_probe(buf, nbytes, sink, stream):
    return lib().moe_read_probe(buf, nbytes, sink, stream)


def moe_route(h, x, T, topk_idx, topk_w, offsets, perm, stream):
    return lib().moe_route(h, x, T, topk_idx, topk_w, offsets, perm, stream)


def moe_forward(h, x, T, y, stream):
    return lib().moe_forward(h, x, T, y, stream)


def moe_forward_host(h, x_host, T, y_host, stream):
    return lib().moe_forward_host(h, x_host, T, y_host, stream)


def moe_get_device_error(h, stream):
    return lib().moe_get_device_error(h, stream)


def moe_destroy(h):
    return lib().moe_destroy(h)


def moe_status_string(status):
    return lib().moe_status_string(status).decode()


def moe_last_cuda_error():
    return lib().moe_last_cuda_error()


def moe_route_one_noalloc(x, d, w_router, router_bias, topk_idx, topk_w, stream):
    """Routing of one token with no device allocation (see include/moe.h)."""
    return lib().moe_route_one_noalloc(x, d, w_router, router_bias, topk_idx, topk_w, stream)


def moe_check_routing(topk_idx, offsets, perm, T, status, stream):
    """Consistency check of a routing (see include/moe.h); *status (a device int) ends as
    MOE_OK or MOE_ERR_DEVICE once the stream has run."""
    return lib().moe_check_routing(topk_idx, offsets, perm, T, status, stream)


def gdn_scan(q, k, v, alpha, beta, state_in, state_out, o, T, H, dk, dv, stream):
    """Gated DeltaNet recurrent scan over T tokens of H heads (see include/gdn.h); device
    pointers, state_in may be None (zero state)."""
    return lib().gdn_scan(q, k, v, alpha, beta, state_in, state_out, o, T, H, dk, dv, stream)


def attn_create(cfg):
    """Returns (status, handle)."""
    h = _c_void_p()
    st = lib().attn_create(ctypes.byref(cfg), ctypes.byref(h))
    return st, h


def attn_destroy(h):
    return lib().attn_destroy(h)


def attn_get_device_error(h, stream):
    return lib().attn_get_device_error(h, stream)


def attn_plan(h, block_table, table_width, ctx_lens, new_lens, B, free_pages, n_free, cursor, T,
              q_offsets, kv_lens, positions, slots, cursor_out, stream):
    return lib().attn_plan(h, block_table, table_width, ctx_lens, new_lens, B, free_pages, n_free,
                           cursor, T, q_offsets, kv_lens, positions, slots, cursor_out, stream)


def attn_qk_norm_rope(h, q, q_stride, k, k_stride, positions, q_weight, k_weight, eps, cos_sin,
                      n_positions, rotary_dim, interleaved, T, q_out, q_out_stride, k_out,
                      k_out_stride, stream):
    return lib().attn_qk_norm_rope(h, q, q_stride, k, k_stride, positions, q_weight, k_weight,
                                   eps, cos_sin, n_positions, rotary_dim, interleaved, T, q_out,
                                   q_out_stride, k_out, k_out_stride, stream)


def attn_kv4_append(h, k, k_stride, v, v_stride, slots, T, cache, stream):
    return lib().attn_kv4_append(h, k, k_stride, v, v_stride, slots, T, cache, stream)


def attn_kv4_read(h, cache, slots, T, k, k_stride, v, v_stride, stream):
    return lib().attn_kv4_read(h, cache, slots, T, k, k_stride, v, v_stride, stream)


def attn_kv4_forward(h, q, q_stride, cache, block_table, table_width, q_offsets, kv_lens, B, T,
                     max_q_len, max_kv_len, out, out_stride, stream):
    return lib().attn_kv4_forward(h, q, q_stride, cache, block_table, table_width, q_offsets,
                                  kv_lens, B, T, max_q_len, max_kv_len, out, out_stride, stream)


def moe_test_expire_waits(h, n_calls):
    """Test hook: the next n_calls batch-1 forwards time out at their grid barrier (see
    include/moe.h)."""
    return lib().moe_test_expire_waits(h, n_calls)


def moe_profile_begin(h, n_calls):
    return lib().moe_profile_begin(h, n_calls)


def moe_profile_end(h):
    """Returns (status, [ms per kernel summed over the recorded calls], n_calls)."""
    ms = (ctypes.c_float * 8)()
    nk, nc = _c_int(), _c_int()
    st = lib().moe_profile_end(h, ms, 8, ctypes.byref(nk), ctypes.byref(nc))
    return st, list(ms)[:nk.value], nc.value


class MoeError(RuntimeError):
    def __init__(self, status, what):
        detail = moe_status_string(status)
        if status == MOE_ERR_CUDA:
            detail += f" (cudaError {moe_last_cuda_error()})"
        super().__init__(f"{what}: {detail}")
        self.status = status


def _check(status, what):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


class MoeLayer:
    """One MoE layer over torch CUDA tensors (bf16 weights, layouts as in include/moe.h).

    weights: dict with w_router [E][d], w_gate/w_up [E][f][d], w_down [E][d][f],
    ws_gate/ws_up [fs][d], ws_down [d][fs] (bf16, contiguous, on the current device) and
    optionally router_bias [E] (float32).  The tensors are borrowed: keep them alive.
    """

    def __init__(self, weights, max_tokens, schedule=MOE_SCHEDULE_AUTO, chunk_tokens=0):
        if isinstance(weights["w_gate"], tuple):
            self._init_q4(weights, max_tokens, schedule, chunk_tokens)
            return
        E, f, d = weights["w_gate"].shape
        fs = weights["ws_gate"].shape[0]
        self.d, self.f, self.fs, self.E, self.k = d, f, fs, E, 8
        self.max_tokens = max_tokens
        self._weights = weights  # keep the borrowed tensors alive
        cfg = moe_config(d, E, 8, f, fs, max_tokens, schedule, chunk_tokens)
        w = moe_weights(_ptr(weights["w_router"]), _ptr(weights.get("router_bias")),
                        _ptr(weights["w_gate"]), _ptr(weights["w_up"]), _ptr(weights["w_down"]),
                        _ptr(weights["ws_gate"]), _ptr(weights["ws_up"]),
                        _ptr(weights["ws_down"]))
        st, self.handle = moe_create(cfg, w)
        _check(st, "moe_create")

    def _init_q4(self, weights, max_tokens, schedule, chunk_tokens):
        """4-bit experts: each expert tensor is a (codes uint8, scales bf16, biases bf16)
        triple of torch tensors, shapes as in synth.q4_shapes; w_router stays bf16."""
        codes = weights["w_gate"][0]
        E, f, d = codes.shape[0], codes.shape[1], codes.shape[2] * 2
        fs = weights["ws_gate"][0].shape[0]
        self.d, self.f, self.fs, self.E, self.k = d, f, fs, E, 8
        self.max_tokens = max_tokens
        self._weights = weights

        def m(name):
            c, sc, b = weights[name]
            return moe_q4_matrix(_ptr(c), _ptr(sc), _ptr(b))

        cfg = moe_config(d, E, 8, f, fs, max_tokens, schedule, chunk_tokens)
        w = moe_weights_q4(_ptr(weights["w_router"]), _ptr(weights.get("router_bias")),
                           m("w_gate"), m("w_up"), m("w_down"), m("ws_gate"), m("ws_up"),
                           m("ws_down"))
        st, self.handle = moe_create_q4(cfg, w)
        _check(st, "moe_create_q4")

    @staticmethod
    def _stream(stream):
        import torch
        s = torch.cuda.current_stream() if stream is None else stream
        return s.cuda_stream

    def forward(self, x, y=None, stream=None):
        import torch
        T = x.shape[0]
        if y is None and stream is None:
            y = torch.empty_like(x)
        elif y is None:
            with torch.cuda.stream(stream):  # memory of the stream that writes it
                y = torch.empty_like(x)
        _check(moe_forward(self.handle, _ptr(x), T, _ptr(y), self._stream(stream)), "moe_forward")
        return y

    def forward_host(self, x_host, y_host, stream=None):
        _check(moe_forward_host(self.handle, _ptr(x_host), x_host.shape[0], _ptr(y_host),
                                self._stream(stream)), "moe_forward_host")
        return y_host

    def route(self, x, stream=None):
        import torch
        T = x.shape[0]
        dev = x.device
        with torch.cuda.stream(stream):
            out = dict(topk_idx=torch.empty((T, 8), dtype=torch.int32, device=dev),
                       topk_w=torch.empty((T, 8), dtype=torch.float32, device=dev),
                       offsets=torch.empty(self.E + 1, dtype=torch.int32, device=dev),
                       perm=torch.empty(T * 8, dtype=torch.int32, device=dev))
        _check(moe_route(self.handle, _ptr(x), T, _ptr(out["topk_idx"]), _ptr(out["topk_w"]),
                         _ptr(out["offsets"]), _ptr(out["perm"]), self._stream(stream)),
               "moe_route")
        return out

    def device_error(self, stream=None):
        return moe_get_device_error(self.handle, self._stream(stream))

    def close(self):
        if self.handle:
            _check(moe_destroy(self.handle), "moe_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _refuse(status, what):
    raise MoeError(status, what)


def _missing(what):
    _refuse(MOE_ERR_INVALID_ARG, f"{what}: missing")


class Kv4Cache:
    """One layer's 4-bit cache as a torch tensor of records [n_pages][Hkv][page_size / 16][bytes]
    (layout in include/attn.h)."""

    def __init__(self, n_pages, n_kv_heads, page_size, head_dim, device="cuda"):
        import torch
        self.data = torch.zeros((n_pages, n_kv_heads, page_size // 16, 18 * head_dim),
                                dtype=torch.uint8, device=device)
        self.layout = (n_pages, n_kv_heads, page_size, head_dim)

    @property
    def ptr(self):
        return self.data.data_ptr()


class PagedAttention:
    """The attention step over a paged 4-bit cache (include/attn.h) on torch CUDA tensors.

    One object serves every layer of the same shape; each layer has a cache of its own
    (new_cache).  Queries, keys, values and outputs are bf16 [T][heads][head_dim], rows may be
    strided (views of a fused projection's output).  Calls are enqueued on the current stream, or
    on `stream`.  Outputs not given are allocated as memory of that stream: another one that uses
    them waits for it first, and has them recorded (Tensor.record_stream) if they may be freed
    before it is done.  The object belongs to the device that was current when it was made: tensors
    are on that device, and calls are made while it is current.
    """

    def __init__(self, n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_requests,
                 scale=0.0):
        import torch
        self.handle = None
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.page_size, self.n_pages, self.max_requests = page_size, n_pages, max_requests
        self._layout = (n_pages, n_kv_heads, page_size, head_dim)
        cfg = attn_config(n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_requests,
                          scale)
        st, self.handle = attn_create(cfg)
        _check(st, "attn_create")
        self._lib = lib()
        self._device = torch.cuda.current_device()
        self._bf16, self._i32, self._f32 = torch.bfloat16, torch.int32, torch.float32
        self._torch = torch
        # the current stream's handle without a Stream object (3 us a call), where torch has it
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        # (where there is one device no other can be current)
        self._current_device = (None if torch.cuda.device_count() == 1 else
                                getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device))

    def new_cache(self):
        return Kv4Cache(self.n_pages, self.n_kv_heads, self.page_size, self.head_dim,
                        f"cuda:{self._device}")

    def _stream(self, stream):
        device = self._device
        if self._current_device is not None and self._current_device() != device:
            self._elsewhere()
        if stream is not None:
            if stream.device_index != device:
                self._elsewhere()
            return stream.cuda_stream
        if self._raw_stream is not None:
            return self._raw_stream(device)
        return self._torch.cuda.current_stream(device).cuda_stream

    def _elsewhere(self):
        _refuse(MOE_ERR_INVALID_ARG, f"expected cuda:{self._device}, the device of this object, "
                "to be current, and a stream of it")

    def _rows(self, t, what, heads, tokens):
        """(address, token stride) of bf16 rows [tokens][heads][head_dim]."""
        if t is None:
            _missing(what)
        D = self.head_dim
        shape, stride = t.shape, t.stride()
        if (t.dtype is not self._bf16 or t.get_device() != self._device
                or shape != (tokens, heads, D)):
            _refuse(MOE_ERR_INVALID_ARG, f"{what}: expected a bfloat16 tensor of shape "
                    f"{(tokens, heads, D)} on cuda:{self._device}, got {t.dtype} {tuple(shape)} on "
                    f"{t.device}")
        if stride[2] != 1 or (heads > 1 and stride[1] != D):
            _refuse(MOE_ERR_UNSUPPORTED, f"{what}: a token's heads must be contiguous")
        # with one token the stride says nothing
        return t.data_ptr(), stride[0] if tokens > 1 else heads * D

    def _ints(self, t, what, n):
        """Address of n contiguous int32 numbers."""
        if t is None:
            _missing(what)
        if (t.dtype is not self._i32 or t.get_device() != self._device or t.numel() != n
                or not t.is_contiguous()):
            _refuse(MOE_ERR_INVALID_ARG, f"{what}: expected {n} contiguous int32 numbers on "
                    f"cuda:{self._device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _cache(self, cache):
        if cache is None:
            _missing("cache")
        data = cache.data
        if cache.layout != self._layout or data.get_device() != self._device:
            _refuse(MOE_ERR_INVALID_ARG, f"cache: expected (pages, heads, page, channels) "
                    f"{self._layout} on cuda:{self._device}, got {cache.layout} on "
                    f"{data.device}")
        return data.data_ptr()

    def _new(self, shape, dtype, stream):
        if stream is None:
            return self._torch.empty(shape, dtype=dtype, device=f"cuda:{self._device}")
        with self._torch.cuda.stream(stream):
            return self._torch.empty(shape, dtype=dtype, device=f"cuda:{self._device}")

    def plan(self, block_table, ctx_lens, new_lens, free_pages, cursor, q_offsets=None,
             kv_lens=None, positions=None, slots=None, cursor_out=None, T=None, stream=None):
        """Extends block_table for new_lens tokens after ctx_lens cached ones, taking pages from
        free_pages[cursor:]; returns (q_offsets, kv_lens, positions, slots, cursor_out).  Without
        positions, T gives the capacity of positions and slots."""
        if block_table is None or free_pages is None:
            _missing("block_table" if block_table is None else "free_pages")
        B, width = block_table.shape
        i32 = self._i32
        if positions is not None:
            T = positions.numel()
        elif T is None:
            _refuse(MOE_ERR_INVALID_ARG, "plan: positions or T")
        else:
            positions = self._new(T, i32, stream)
        slots = self._new(T, i32, stream) if slots is None else slots
        q_offsets = self._new(B + 1, i32, stream) if q_offsets is None else q_offsets
        kv_lens = self._new(B, i32, stream) if kv_lens is None else kv_lens
        cursor_out = self._new(1, i32, stream) if cursor_out is None else cursor_out
        ints = self._ints
        n_free = free_pages.numel()
        st = self._lib.attn_plan(
            self.handle, ints(block_table, "block_table", B * width), width,
            ints(ctx_lens, "ctx_lens", B), ints(new_lens, "new_lens", B), B,
            ints(free_pages, "free_pages", n_free), n_free, ints(cursor, "cursor", 1), T,
            ints(q_offsets, "q_offsets", B + 1), ints(kv_lens, "kv_lens", B),
            ints(positions, "positions", T), ints(slots, "slots", T),
            ints(cursor_out, "cursor_out", 1), self._stream(stream))
        if st:
            _check(st, "attn_plan")
        return q_offsets, kv_lens, positions, slots, cursor_out

    def qk_norm_rope(self, q, k, positions, q_weight, k_weight, cos_sin, eps=1e-6,
                     interleaved=False, q_out=None, k_out=None, stream=None):
        """Norm of each query and key head and rotation by cos_sin [positions][rotary_dim] (None:
        no rotation, and positions may be None); returns (q_out, k_out)."""
        if q is None or q_weight is None or k_weight is None:
            _missing("q, q_weight or k_weight")
        T, Hq, Hkv, D = q.shape[0], self.n_q_heads, self.n_kv_heads, self.head_dim
        q_out = self._new((T, Hq, D), self._bf16, stream) if q_out is None else q_out
        k_out = self._new((T, Hkv, D), self._bf16, stream) if k_out is None else k_out
        rows = self._rows
        (qp, qs), (kp, ks) = rows(q, "q", Hq, T), rows(k, "k", Hkv, T)
        (qop, qos), (kop, kos) = rows(q_out, "q_out", Hq, T), rows(k_out, "k_out", Hkv, T)
        for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if (w.dtype is not self._bf16 or w.get_device() != self._device or w.shape != (D,)
                    or w.stride(0) != 1):
                _refuse(MOE_ERR_INVALID_ARG, f"{what}: expected {D} contiguous bfloat16 on "
                        f"cuda:{self._device}")
        n_pos = rot = 0
        pos = table = None
        if cos_sin is not None:
            if (cos_sin.dtype is not self._f32 or cos_sin.get_device() != self._device
                    or cos_sin.dim() != 2 or not cos_sin.is_contiguous()):
                _refuse(MOE_ERR_INVALID_ARG, "cos_sin: expected a contiguous float32 matrix on "
                        f"cuda:{self._device}")
            n_pos, rot = cos_sin.shape
            pos, table = self._ints(positions, "positions", T), cos_sin.data_ptr()
        st = self._lib.attn_qk_norm_rope(
            self.handle, qp, qs, kp, ks, pos, q_weight.data_ptr(), k_weight.data_ptr(), eps,
            table, n_pos, rot, 1 if interleaved else 0, T, qop, qos, kop, kos,
            self._stream(stream))
        if st:
            _check(st, "attn_qk_norm_rope")
        return q_out, k_out

    def append(self, k, v, slots, cache, stream=None):
        """Quantises keys and values [T][Hkv][D] into the cached rows of slots [T]."""
        if k is None:
            _missing("k")
        T, Hkv = k.shape[0], self.n_kv_heads
        (kp, ks), (vp, vs) = self._rows(k, "k", Hkv, T), self._rows(v, "v", Hkv, T)
        st = self._lib.attn_kv4_append(self.handle, kp, ks, vp, vs,
                                       self._ints(slots, "slots", T), T, self._cache(cache),
                                       self._stream(stream))
        if st:
            _check(st, "attn_kv4_append")

    def read(self, slots, cache, k_out=None, v_out=None, stream=None):
        """Cached rows of slots [T] as bf16; returns (k_out, v_out)."""
        if slots is None:
            _missing("slots")
        T, Hkv = slots.shape[0], self.n_kv_heads
        k_out = self._new((T, Hkv, self.head_dim), self._bf16, stream) if k_out is None else k_out
        v_out = self._new((T, Hkv, self.head_dim), self._bf16, stream) if v_out is None else v_out
        (kp, ks), (vp, vs) = self._rows(k_out, "k_out", Hkv, T), self._rows(v_out, "v_out", Hkv, T)
        st = self._lib.attn_kv4_read(self.handle, self._cache(cache),
                                     self._ints(slots, "slots", T), T, kp, ks, vp, vs,
                                     self._stream(stream))
        if st:
            _check(st, "attn_kv4_read")
        return k_out, v_out

    def forward(self, q, cache, block_table, q_offsets, kv_lens, max_q_len, max_kv_len, out=None,
                stream=None):
        """Causal attention of the requests' new tokens over their cached rows; returns out."""
        if q is None or block_table is None:
            _missing("q" if q is None else "block_table")
        T, Hq = q.shape[0], self.n_q_heads
        B, width = block_table.shape
        out = self._new((T, Hq, self.head_dim), self._bf16, stream) if out is None else out
        (qp, qs), (op, os_) = self._rows(q, "q", Hq, T), self._rows(out, "out", Hq, T)
        ints = self._ints
        st = self._lib.attn_kv4_forward(
            self.handle, qp, qs, self._cache(cache), ints(block_table, "block_table", B * width),
            width, ints(q_offsets, "q_offsets", B + 1), ints(kv_lens, "kv_lens", B), B, T,
            max_q_len, max_kv_len, op, os_, self._stream(stream))
        if st:
            _check(st, "attn_kv4_forward")
        return out

    def device_error(self, stream=None):
        return attn_get_device_error(self.handle, self._stream(stream))

    def close(self):
        if self.handle:
            with self._torch.cuda.device(self._device):
                _check(attn_destroy(self.handle), "attn_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
