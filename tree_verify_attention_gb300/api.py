"""Thin Python binding of libdfv (include/dfv.h) over torch device tensors.

PyTorch provides device memory and streams only; each function checks
dtypes/shapes, passes raw pointers to the C ABI and raises DfvError on a
non-OK status. No compute happens here.
"""

import ctypes
import decimal
import math

import torch

from . import _lib

DTYPE_F32 = 0
DTYPE_BF16 = 1
KV_F16 = 1
KV_Q4_0 = 2
KV_TREE_AS_CACHE = 0x100
STEP_PIPELINED = 0x200
_FORMATS = {"q4_0": KV_Q4_0, "f16": KV_F16}
MAX_NODES = 65
MASK_WORDS = (MAX_NODES + 31) // 32

DEV_BAD_TREE = 0x1
DEV_DEPTH = 0x2
DEV_CAPACITY = 0x4
DEV_CTX = 0x8
DEV_BAD_PATH = 0x10
DEV_TIMEOUT = 0x20
DEV_NONFINITE = 0x40
DEV_BAD_TOKEN = 0x80
DEV_BAD_SAMPLING = 0x100
MAX_SAMPLE_VOCAB = 1 << 19

KV8_BLOCK = 64       # positions that share a scale in an Int8Cache
MAX_TOP = 32         # alternatives token_logprobs can return


class DfvError(RuntimeError):
    pass


def lib():
    return _lib.load()


def _check(st, name):
    if st != 0:
        msg = lib().dfv_status_string(st).decode()
        raise DfvError(f"{name}: {msg} (status {st})")


def _stream(stream, index=None):
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle without building a Stream object (2 us a call)
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if index is None else index)


def _p(t):
    return None if t is None else t.data_ptr()


def _dev(t, name, dtypes, numel=None):
    if (t is not None and t.dtype in dtypes and t.is_cuda and t.is_contiguous()
            and (numel is None or t.numel() >= numel)):
        return t
    if t is None:
        raise DfvError(f"{name} is required")
    if not t.is_cuda or not t.is_contiguous():
        raise DfvError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype not in dtypes:
        raise DfvError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if numel is not None and t.numel() < numel:
        raise DfvError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t


def _ptr(t, name, dtype, numel, index):
    """Address of a contiguous tensor of ``dtype`` on device ``index`` with at
    least ``numel`` elements; None for None."""
    if t is None:
        return None
    if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
            and t.numel() >= numel):
        return t.data_ptr()
    _dev(t, name, (dtype,), numel)
    raise DfvError(f"{name} is on {t.device}, expected cuda:{index}")


_BF16 = (torch.bfloat16, torch.int16)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def q4_0_row_bytes(head_dim):
    return head_dim // 32 * 18


def row_bytes(head_dim, fmt="q4_0"):
    """Bytes of one cache row (one KV head, one position)."""
    if fmt == "f16":
        return head_dim * 2
    return q4_0_row_bytes(head_dim)


def _fmt_code(fmt):
    if fmt not in _FORMATS:
        raise DfvError(f"unknown cache format {fmt!r} (expected one of {sorted(_FORMATS)})")
    return _FORMATS[fmt]


class KVCache:
    """Device KV cache of one sequence in format ``fmt`` ("q4_0" or "f16"):
    K and V byte tensors [Hkv, capacity, row bytes], the committed length
    (device int32), and ``dropped``, the number of positions by which its rows
    lie below their place in the sequence (device int32; 0 until
    :func:`kv_evict` has moved rows into it, and again after a :meth:`fill` from
    position 0; who sets ``ctx_len`` back by hand sets it back too)."""

    def __init__(self, n_kv_heads, head_dim, capacity, device="cuda", fmt="q4_0"):
        self.n_kv_heads, self.head_dim, self.capacity = n_kv_heads, head_dim, capacity
        self.fmt = fmt
        self.kv_format = _fmt_code(fmt)
        shape = (n_kv_heads, capacity, row_bytes(head_dim, fmt))
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.ctx_len = torch.zeros(1, dtype=torch.int32, device=device)
        self.dropped = torch.zeros(1, dtype=torch.int32, device=device)

    def fill(self, k_rows, v_rows, pos0=0, stream=None):
        """Encode float rows [Hkv, n, D] (f32 or bf16) into positions
        [pos0, pos0 + n) and set the committed length to pos0 + n. With pos0 =
        0 another sequence begins: ``dropped`` is 0 again."""
        n = k_rows.shape[1]
        for src, dst in ((k_rows, self.k), (v_rows, self.v)):
            kv_quantize_rows(dst, src, pos0, self.n_kv_heads, self.head_dim, self.capacity,
                             head_major=True, stream=stream, fmt=self.fmt)
        with torch.cuda.stream(stream):   # (None: the current one)
            self.ctx_len.fill_(pos0 + n)
            if pos0 == 0:
                self.dropped.zero_()

    def read(self, pos0, n, k_out, v_out, head_major=False, stream=None):
        """The values of rows [pos0, pos0 + n) into k_out and v_out, [n, Hkv,
        D] (or [Hkv, n, D]) f32 or bf16 with equal strides."""
        h, d = self.n_kv_heads, self.head_dim
        r, hd = (1, 0) if head_major else (0, 1)
        shape = (h, n, d) if head_major else (n, h, d)
        if not 0 <= pos0 <= pos0 + n <= self.capacity:
            raise DfvError(f"rows [{pos0}, {pos0 + n}) are outside [0, {self.capacity})")
        st = _float_rows(k_out, "k_out", shape)
        if _float_rows(v_out, "v_out", shape, (k_out.dtype,)) != st:
            raise DfvError("k_out and v_out must have the same strides")
        index = self.k.get_device()
        if (index != torch._C._cuda_getDevice() or k_out.get_device() != index
                or v_out.get_device() != index):
            _same_device(index, k_out, v_out)
        _check(lib().dfv_kv_read_rows(
            h, d, self.kv_format, self.capacity, pos0, n, self.k.data_ptr(), self.v.data_ptr(),
            k_out.data_ptr(), v_out.data_ptr(),
            DTYPE_F32 if k_out.dtype is torch.float32 else DTYPE_BF16, st[r], st[hd],
            _stream(stream, index)), "dfv_kv_read_rows")


class Q4Cache(KVCache):
    """Device Q4_0 KV cache of one sequence: K and V byte tensors
    [Hkv, capacity, D/32 * 18] and the committed length (device int32)."""

    def __init__(self, n_kv_heads, head_dim, capacity, device="cuda"):
        super().__init__(n_kv_heads, head_dim, capacity, device=device, fmt="q4_0")


def _same_device(index, *tensors):
    """All of ``tensors`` (None allowed) on device ``index``, which is the
    current one: the library launches on the current device."""
    if index != torch.cuda.current_device():
        raise DfvError(f"tensors on cuda:{index}, but the current device is "
                       f"cuda:{torch.cuda.current_device()}")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise DfvError(f"a tensor is on {t.device}, expected cuda:{index}")


_ROWS = (torch.float32, torch.bfloat16)


def _float_rows(t, name, shape, dtypes=_ROWS):
    if t is None or not t.is_cuda or t.dtype not in dtypes:
        raise DfvError(f"{name} must be a CUDA f32 or bf16 tensor")
    if t.shape != shape:
        raise DfvError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    st = t.stride()
    if st[-1] != 1 and t.numel():
        raise DfvError(f"{name} rows must be contiguous")
    return st


class Int8Cache:
    """Device KV cache of one sequence held in 8 bits: signed codes with one
    float32 scale for each block of 64 positions and head; the open block and
    the one before it are also kept as bf16 rows (``k_tail``, ``v_tail``), so a
    block is quantised once, when it is complete. The layouts are those of
    ``dfv_kv8_cache`` (include/dfv.h).

    Every method is asynchronous on ``stream`` (the current one by default);
    problems that only the device can see are OR-ed into ``status`` (int32[1],
    DEV_* bits; :attr:`status` of the cache by default). After DEV_TIMEOUT from
    a write, later writes are refused until ``state[3]`` is zeroed; rows from
    the start of the write that gave up have to be written again."""

    fmt = "int8"

    def __init__(self, n_kv_heads, head_dim, capacity, device="cuda"):
        if head_dim not in (64, 128, 256):
            raise DfvError(f"head_dim {head_dim} is not one of 64, 128, 256")
        if not (1 <= n_kv_heads <= 65535 and 1 <= capacity <= 1 << 30):
            raise DfvError(f"bad cache shape ({n_kv_heads} heads, capacity {capacity})")
        self.n_kv_heads, self.head_dim, self.capacity = n_kv_heads, head_dim, capacity
        nblk = -(-capacity // KV8_BLOCK)
        h, d = n_kv_heads, head_dim
        # nothing is read of a block before it is complete: no need to clear
        self.k = torch.empty(h, nblk, d // 16, KV8_BLOCK, 16, dtype=torch.int8, device=device)
        self.v = torch.empty(h, nblk, KV8_BLOCK // 16, d, 16, dtype=torch.int8, device=device)
        self.k_scale = torch.empty(h, nblk, device=device)
        self.v_scale = torch.empty(h, nblk, device=device)
        # the open end in one buffer: a copy of it (and copying it back) saves
        # and restores a point to which the cache can return
        tail = h * 2 * KV8_BLOCK * d
        self.open_end = torch.zeros(128 + 4 * tail, dtype=torch.uint8, device=device)
        self.state = self.open_end[:16].view(torch.int32)
        self.k_tail, self.v_tail = (
            self.open_end[128 + 2 * i * tail:128 + 2 * (i + 1) * tail].view(torch.bfloat16)
            .view(h, 2, KV8_BLOCK, d) for i in range(2))
        self.ctx_len = self.state[:1]
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self._struct = _lib.Kv8CacheStruct(
            h, d, capacity, 0, self.state.data_ptr(), self.k.data_ptr(), self.v.data_ptr(),
            self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.k_tail.data_ptr(),
            self.v_tail.data_ptr())
        self.handle = ctypes.addressof(self._struct)
        self._index = self.state.get_device()
        self._status_ptr = self.status.data_ptr()

    def append(self, k_rows, v_rows, at=None, head_major=False, stream=None, status=None):
        """Write float rows [n, Hkv, D] (or [Hkv, n, D] with head_major=True;
        f32 or bf16, last axis contiguous) at positions [at, at + n), and set
        the committed length to at + n. ``at=None`` appends at the committed
        length. An ``at`` behind that length, or inside a block whose bf16
        rows are no longer held, writes nothing and sets DEV_CTX."""
        h, d = self.n_kv_heads, self.head_dim
        r, hd = (1, 0) if head_major else (0, 1)
        n = k_rows.shape[r]
        shape = (h, n, d) if head_major else (n, h, d)
        if at is not None and not 0 <= at <= self.capacity:
            raise DfvError(f"at {at} is outside [0, {self.capacity}]")
        ks = _float_rows(k_rows, "k_rows", shape)
        vs = _float_rows(v_rows, "v_rows", shape, (k_rows.dtype,))
        _same_device(self._index, k_rows, v_rows, status)
        _check(lib().dfv_kv8_append(
            self.handle, -1 if at is None else at, n, k_rows.data_ptr(), v_rows.data_ptr(),
            DTYPE_F32 if k_rows.dtype == torch.float32 else DTYPE_BF16, ks[r], ks[hd], vs[r],
            vs[hd], self._status_ptr if status is None else status.data_ptr(),
            _stream(stream, self._index)), "dfv_kv8_append")

    def fill(self, k_rows, v_rows, pos0=0, stream=None):
        """Rows [Hkv, n, D] at positions [pos0, pos0 + n), as KVCache.fill."""
        self.append(k_rows, v_rows, at=pos0, head_major=True, stream=stream)

    def truncate(self, length, stream=None, status=None):
        """Set the committed length back to ``length`` (the same rule as
        :meth:`append`'s ``at``: 64 rows can always be taken back after a
        write, more if the open block has rows, and any multiple of 64)."""
        none = self.k_tail.new_empty(0, self.n_kv_heads, self.head_dim)
        self.append(none, none, at=length, stream=stream, status=status)

    def read(self, pos0, n, k_out, v_out, head_major=False, stream=None, status=None):
        """The values of rows [pos0, pos0 + n) into k_out and v_out, [n, Hkv,
        D] (or [Hkv, n, D]) f32 or bf16 with equal strides. Rows behind the
        committed length are left as they were (DEV_CTX)."""
        h, d = self.n_kv_heads, self.head_dim
        r, hd = (1, 0) if head_major else (0, 1)
        shape = (h, n, d) if head_major else (n, h, d)
        if not 0 <= pos0 <= pos0 + n <= self.capacity:
            raise DfvError(f"rows [{pos0}, {pos0 + n}) are outside [0, {self.capacity})")
        st = _float_rows(k_out, "k_out", shape)
        if _float_rows(v_out, "v_out", shape, (k_out.dtype,)) != st:
            raise DfvError("k_out and v_out must have the same strides")
        _same_device(self._index, k_out, v_out, status)
        _check(lib().dfv_kv8_read(
            self.handle, pos0, n, k_out.data_ptr(), v_out.data_ptr(),
            DTYPE_F32 if k_out.dtype == torch.float32 else DTYPE_BF16, st[r], st[hd],
            self._status_ptr if status is None else status.data_ptr(),
            _stream(stream, self._index)), "dfv_kv8_read")


def int8_attn_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity):
    return lib().dfv_kv8_attn_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window,
                                              capacity)


def _int8_attn(cache, q, tree_k, tree_v, parent, window, max_depth, out, lse, ws, scale, status,
               stream):
    n, hq, d = q.shape
    hkv = cache.n_kv_heads
    if d != cache.head_dim:
        raise DfvError(f"q has head_dim {d}, the cache {cache.head_dim}")
    _dev(q, "q", _BF16)
    for t, name in ((tree_k, "tree_k"), (tree_v, "tree_v")):
        _dev(t, name, _BF16)
        if t.shape != (n, hkv, d):
            raise DfvError(f"{name} has shape {tuple(t.shape)}, expected {(n, hkv, d)}")
    _dev(parent, "parent", _I32, n)
    _dev(out, "out", _ROWS, n * hq * d)
    if lse is not None:
        _dev(lse, "lse", _F32, n * hq)
    _dev(ws, "workspace", (torch.uint8,))
    _same_device(cache._index, q, tree_k, tree_v, parent, out, lse, ws, status)
    _check(lib().dfv_kv8_attn(
        cache.handle, n, max_depth, hq, window, q.data_ptr(), tree_k.data_ptr(),
        tree_v.data_ptr(), parent.data_ptr(), float(scale), out.data_ptr(),
        DTYPE_F32 if out.dtype == torch.float32 else DTYPE_BF16, _p(lse), ws.data_ptr(),
        ws.numel(), cache._status_ptr if status is None else status.data_ptr(),
        _stream(stream, cache._index)), "dfv_kv8_attn")


def kv_quantize_rows(cache, src, pos0, n_kv_heads, head_dim, capacity, head_major=False,
                     stream=None, fmt="q4_0"):
    """Encode rows of ``src`` into ``cache`` positions [pos0, pos0 + n) in
    format ``fmt`` ("q4_0" or "f16").
    ``src`` is [n, Hkv, D] (or [Hkv, n, D] with head_major=True), f32 or
    bf16, last axis contiguous."""
    if src.dtype not in (torch.float32, torch.bfloat16) or not src.is_cuda:
        raise DfvError("src must be a CUDA f32 or bf16 tensor")
    if src.stride(-1) != 1:
        raise DfvError("src rows must be contiguous")
    if head_major:
        n, s_row, s_head = src.shape[1], src.stride(1), src.stride(0)
    else:
        n, s_row, s_head = src.shape[0], src.stride(0), src.stride(1)
    dt = DTYPE_F32 if src.dtype == torch.float32 else DTYPE_BF16
    _dev(cache, "cache", (torch.uint8,))
    _check(lib().dfv_kv_quantize_rows(n_kv_heads, head_dim, _fmt_code(fmt), capacity, pos0, n,
                                      src.data_ptr(), dt, s_row, s_head, cache.data_ptr(),
                                      _stream(stream)), "dfv_kv_quantize_rows")


def attn_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity):
    return lib().dfv_tree_verify_attn_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim,
                                                      window, capacity)


def accept_workspace_bytes(n_nodes, vocab):
    return lib().dfv_greedy_accept_workspace_bytes(n_nodes, vocab)


def step_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity, vocab):
    return lib().dfv_verify_step_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim,
                                                 window, capacity, vocab)


def step_launches(n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity):
    return lib().dfv_verify_step_launches(n_nodes, n_q_heads, n_kv_heads, head_dim, window,
                                          capacity)


def workspace(nbytes, device="cuda", stream=None):
    """A zeroed, 256-byte aligned device workspace of ``nbytes``."""
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    _check(lib().dfv_workspace_clear(ws.data_ptr(), ws.numel(), _stream(stream)),
           "dfv_workspace_clear")
    return ws


def clear_workspace(ws, stream=None):
    """Zero a workspace on the device (dfv_workspace_clear): before its first
    use, and again after a step reported DFV_DEV_TIMEOUT."""
    _dev(ws, "workspace", (torch.uint8,))
    _check(lib().dfv_workspace_clear(ws.data_ptr(), ws.numel(), _stream(stream)),
           "dfv_workspace_clear")


def tree_verify_attn(cache, q, tree_k, tree_v, parent, window, max_depth, out, lse, ws,
                     scale=0.0, status=None, stream=None, tree_as_cache=False, pipelined=False):
    """Tree-masked attention over ``cache`` (KVCache, Q4Cache or Int8Cache).
    With an Int8Cache, ``out`` may be f32 or bf16, the workspace comes from
    :func:`int8_attn_workspace_bytes`, and ``tree_as_cache`` and ``pipelined``
    are not available."""
    if isinstance(cache, Int8Cache):
        if tree_as_cache or pipelined:
            raise DfvError("tree_as_cache and pipelined are not available with an Int8Cache")
        return _int8_attn(cache, q, tree_k, tree_v, parent, window, max_depth, out, lse, ws,
                          scale, status, stream)
    n, hq, d = q.shape
    hkv = tree_k.shape[1]
    _dev(q, "q", _BF16)
    _dev(tree_k, "tree_k", _BF16, n * hkv * d)
    _dev(tree_v, "tree_v", _BF16, n * hkv * d)
    _dev(parent, "parent", _I32, n)
    _dev(out, "out", _F32, n * hq * d)
    if lse is not None:
        _dev(lse, "lse", _F32, n * hq)
    kvf = (cache.kv_format | (KV_TREE_AS_CACHE if tree_as_cache else 0)
           | (STEP_PIPELINED if pipelined else 0))
    _check(lib().dfv_tree_verify_attn(
        n, max_depth, hq, hkv, d, window, kvf, cache.capacity, cache.ctx_len.data_ptr(),
        cache.k.data_ptr(), cache.v.data_ptr(), q.data_ptr(), tree_k.data_ptr(),
        tree_v.data_ptr(), parent.data_ptr(), float(scale), out.data_ptr(), _p(lse),
        ws.data_ptr(), ws.numel(), _p(status), _stream(stream)), "dfv_tree_verify_attn")


def build_tree_mask(parent, depth, anc_mask, status=None, stream=None):
    """depth [N] (int32) and ancestor-or-self bitmasks [N, MASK_WORDS]
    (int32 tensor holding the uint32 words) of the tree given by ``parent``."""
    n = parent.numel()
    _dev(parent, "parent", _I32, n)
    _dev(depth, "depth", _I32, n)
    _dev(anc_mask, "anc_mask", _I32, n * MASK_WORDS)
    _check(lib().dfv_build_tree_mask(n, parent.data_ptr(), depth.data_ptr(), anc_mask.data_ptr(),
                                     _p(status), _stream(stream)), "dfv_build_tree_mask")


def greedy_accept(logits, parent, tokens, argmax, accept_len, path, out_tokens, ws,
                  status=None, stream=None):
    n, vocab = logits.shape
    dt = DTYPE_F32 if logits.dtype == torch.float32 else DTYPE_BF16
    _dev(logits, "logits", (torch.float32,) + _BF16)
    for t, nm in ((parent, "parent"), (tokens, "tokens"), (argmax, "argmax"), (path, "path"),
                  (out_tokens, "out_tokens")):
        _dev(t, nm, _I32, n)
    _dev(accept_len, "accept_len", _I32, 1)
    _check(lib().dfv_greedy_accept(
        n, vocab, dt, logits.data_ptr(), parent.data_ptr(), tokens.data_ptr(), argmax.data_ptr(),
        accept_len.data_ptr(), path.data_ptr(), out_tokens.data_ptr(), ws.data_ptr(), ws.numel(),
        _p(status), _stream(stream)), "dfv_greedy_accept")


def token_logprobs(logits, tokens, logprob, entropy=None, top_ids=None, top_logprobs=None,
                   status=None, stream=None):
    """Log probability of ``tokens`` [N] (int32) under each row of ``logits``
    [N, V] (f32 or bf16, rows may be strided) into ``logprob`` [N], the
    entropy of each row into ``entropy`` [N], and its most probable tokens
    into ``top_ids`` / ``top_logprobs`` [N, K], K <= MAX_TOP (either may be
    None). Ties go to the lowest index."""
    if logits is None or not logits.is_cuda or logits.dim() != 2 or \
            logits.dtype not in (torch.float32, torch.bfloat16):
        raise DfvError("logits must be a CUDA f32 or bf16 tensor [N, V]")
    n, vocab = logits.shape
    if n and vocab > 1 and logits.stride(1) != 1:
        raise DfvError("logits rows must be contiguous")
    if logprob is not None:
        _dev(tokens, "tokens", _I32, n)
        _dev(logprob, "logprob", _F32, n)
    if entropy is not None:
        _dev(entropy, "entropy", _F32, n)
    top = None
    for t, name, dt in ((top_ids, "top_ids", _I32), (top_logprobs, "top_logprobs", _F32)):
        if t is None:
            continue
        _dev(t, name, dt)
        if t.dim() != 2 or t.shape[0] != n or t.shape[1] != (t.shape[1] if top is None else top):
            raise DfvError(f"{name} must be [{n}, K], the same K for ids and log probabilities")
        top = t.shape[1]
    top = top or 0
    if top > min(MAX_TOP, vocab):
        raise DfvError(f"{top} alternatives asked for, at most {min(MAX_TOP, vocab)}")
    _same_device(logits.get_device(), tokens, logprob, entropy, top_ids, top_logprobs, status)
    _check(lib().dfv_token_logprobs(
        n, vocab, DTYPE_F32 if logits.dtype == torch.float32 else DTYPE_BF16, logits.data_ptr(),
        logits.stride(0) if n > 1 else vocab, _p(tokens), top, _p(logprob), _p(entropy),
        _p(top_ids), _p(top_logprobs), _p(status), _stream(stream)), "dfv_token_logprobs")


def _kv_cache(cache, name):
    if not isinstance(cache, KVCache):
        raise DfvError(f"{name} must be a KVCache (Q4_0 or F16)")


def kv_weights(cache, q, lse, weights, prev=None, decay=1.0, path=None, accept_len=None, window=0,
               scale=0.0, status=None, stream=None):
    """The attention weight that each key of ``cache`` (a KVCache) receives
    from its last committed rows, into ``weights`` [Hkv, capacity] (f32):
    ``decay * prev`` (zero without, and for the new rows) plus, over the rows
    that see the key and the query heads of its group, exp(scale q . k - lse).
    ``prev`` may be ``weights`` itself.

    ``q`` [N, Hq, D] (bf16) and ``lse`` [N, Hq] are the rows' queries and what
    the attention gave for them; they stand at the last N positions, or, with a
    step's ``path`` and ``accept_len``, its accepted nodes at the last
    ``accept_len`` ones: call it after the commit."""
    _kv_cache(cache, "cache")
    _dev(q, "q", _BF16)
    if q.dim() != 3:
        raise DfvError("q must be [N, Hq, D]")
    n, hq, d = q.shape
    h, cap = cache.n_kv_heads, cache.capacity
    if d != cache.head_dim:
        raise DfvError(f"q has head_dim {d}, the cache {cache.head_dim}")
    for t, name in ((weights, "weights"), (prev, "prev")):
        if t is not None and t.shape != (h, cap):
            raise DfvError(f"{name} has shape {tuple(t.shape)}, expected {(h, cap)}")
    if weights is None or lse is None:
        raise DfvError("weights and lse are required")
    if not 0 <= window < 1 << 31:
        raise DfvError(f"window {window} is out of range")
    index = q.get_device()
    if index != torch._C._cuda_getDevice() or cache.k.get_device() != index:
        _same_device(index, cache.k)
    _check(lib().dfv_kv_weights(
        n, hq, h, d, window, cache.kv_format, cap, cache.ctx_len.data_ptr(), cache.k.data_ptr(),
        q.data_ptr(), _ptr(lse, "lse", torch.float32, n * hq, index),
        _ptr(path, "path", torch.int32, n, index),
        _ptr(accept_len, "accept_len", torch.int32, 1, index), scale, decay,
        _ptr(prev, "prev", torch.float32, 0, index),
        _ptr(weights, "weights", torch.float32, 0, index),
        _ptr(status, "status", torch.int32, 1, index), _stream(stream, index)), "dfv_kv_weights")


def kv_evict(cache, weights, into, kept, sinks=0, recent=0, weights_out=None, status=None,
             stream=None):
    """Move the rows of ``cache`` whose keys have the largest ``weights`` [Hkv,
    capacity] into ``into``, another KVCache of the same heads and format: of
    each head at most K rows, K the width of ``kept`` [Hkv, K] (int32), which
    receives their positions: the first ``sinks``, the last ``recent``, the best
    of the others (ties to the lowest position), in their order. ``into``'s length
    and ``dropped`` follow, and ``weights_out`` [Hkv, into.capacity] receives
    the kept rows' weights."""
    _kv_cache(cache, "cache")
    _kv_cache(into, "into")
    h, d, cap, into_cap = cache.n_kv_heads, cache.head_dim, cache.capacity, into.capacity
    if (into.n_kv_heads, into.head_dim, into.fmt) != (h, d, cache.fmt):
        raise DfvError("into must be a cache of the same heads and format")
    k_src, k_dst, index = cache.k.data_ptr(), into.k.data_ptr(), cache.k.get_device()
    if k_src == k_dst:
        raise DfvError("into must be another cache")
    if index != torch._C._cuda_getDevice() or into.k.get_device() != index:
        _same_device(index, into.k)
    if weights.shape != (h, cap):
        raise DfvError(f"weights has shape {tuple(weights.shape)}, expected {(h, cap)}")
    keep = kept.shape[-1] if kept.dim() == 2 else 0
    if kept.shape != (h, keep) or not 1 <= keep <= into_cap:
        raise DfvError(f"kept must be [{h}, K], K in [1, {into_cap}]")
    if sinks < 0 or recent < 0 or sinks + recent > keep:
        raise DfvError(f"{sinks} first and {recent} last rows of {keep}")
    if weights_out is not None:
        if weights_out.shape != (h, into_cap):
            raise DfvError(f"weights_out has shape {tuple(weights_out.shape)}, expected "
                           f"{(h, into_cap)}")
        if weights_out.data_ptr() == weights.data_ptr():
            raise DfvError("weights_out must not be weights")
    _check(lib().dfv_kv_evict(
        h, d, cache.kv_format, cap, cache.ctx_len.data_ptr(), cache.dropped.data_ptr(), k_src,
        cache.v.data_ptr(), _ptr(weights, "weights", torch.float32, 0, index), keep, sinks,
        recent, into_cap, k_dst, into.v.data_ptr(), into.ctx_len.data_ptr(),
        into.dropped.data_ptr(), _ptr(weights_out, "weights_out", torch.float32, 0, index),
        _ptr(kept, "kept", torch.int32, 0, index),
        _ptr(status, "status", torch.int32, 1, index), _stream(stream, index)), "dfv_kv_evict")


class Sampling:
    """How tokens are drawn: ``temperature``, ``top_k`` (0: off), ``top_p`` (1:
    off) and ``min_p`` (0: off), in this order; each a number for all rows, or a
    device tensor [N] (f32, ``top_k`` int32) with each row's own. Tensors are
    read when a call runs, so their values may change between calls."""

    def __init__(self, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
        self.tensors = []
        values = []
        for x, name, dt in ((temperature, "temperature", _F32), (top_k, "top_k", _I32),
                            (top_p, "top_p", _F32), (min_p, "min_p", _F32)):
            if isinstance(x, torch.Tensor):
                self.tensors.append((_dev(x, name, dt), name))
                values.append((x.data_ptr(), 0))
                continue
            if x != x or (name == "temperature" and not 0 <= x < math.inf):
                raise DfvError(f"{name} {x} is out of range")
            values.append((None, int(max(0, min(x, 2 ** 31 - 1))) if name == "top_k"
                           else float(x)))
        self._struct = _lib.SamplingStruct(*(v[0] for v in values), *(v[1] for v in values))
        self.handle = ctypes.addressof(self._struct)

    def check(self, n, index):
        """That the tensors serve ``n`` rows on device ``index``."""
        for t, name in self.tensors:
            if t.numel() < n:
                raise DfvError(f"{name} holds {t.numel()} elements, needs {n}")
            if t.get_device() != index:
                raise DfvError(f"{name} is on {t.device}, expected cuda:{index}")


def _sample_args(logits, uniform, sampling, token):
    if logits is None or not logits.is_cuda or logits.dim() != 2 or logits.dtype not in _ROWS:
        raise DfvError("logits must be a CUDA f32 or bf16 tensor [N, V]")
    n, vocab = logits.shape
    row, one = logits.stride()
    if one != 1 and n and vocab > 1:
        raise DfvError("logits rows must be contiguous")
    if vocab > MAX_SAMPLE_VOCAB:
        raise DfvError(f"{vocab} logits a row, at most {MAX_SAMPLE_VOCAB}")
    if not isinstance(sampling, Sampling):
        raise DfvError("sampling must be a Sampling")
    index = logits.get_device()
    if index != torch._C._cuda_getDevice():
        _same_device(index)
    if sampling.tensors:
        sampling.check(n, index)
    if uniform is None or token is None:
        raise DfvError("uniform and token are required")
    return (n, vocab, DTYPE_F32 if logits.dtype is torch.float32 else DTYPE_BF16,
            logits.data_ptr(), row if n > 1 else vocab,
            _ptr(uniform, "uniform", torch.float32, n, index), sampling.handle), index


def sample_tokens(logits, uniform, sampling, token, logprob=None, status=None, stream=None):
    """Draw a token from each row of ``logits`` [N, V] (f32 or bf16, rows may
    be strided) by ``sampling`` (:class:`Sampling`) and the random numbers
    ``uniform`` [N] in [0, 1) into ``token`` [N] (int32), and its log probability
    among the tokens that could have been drawn into ``logprob`` [N]. The first
    token in index order is taken at which the running sum of the kept
    probabilities exceeds the random number. A row without a distribution gets
    -1 and NaN (DEV_NONFINITE, DEV_BAD_SAMPLING)."""
    args, index = _sample_args(logits, uniform, sampling, token)
    n = args[0]
    _check(lib().dfv_sample(*args, _ptr(token, "token", torch.int32, n, index),
                            _ptr(logprob, "logprob", torch.float32, n, index),
                            _ptr(status, "status", torch.int32, 1, index),
                            _stream(stream, index)), "dfv_sample")


def sample_accept_workspace_bytes(n_nodes, vocab):
    return lib().dfv_sample_accept_workspace_bytes(n_nodes, vocab)


def sample_accept(logits, uniform, sampling, parent, tokens, target, accept_len, path, out_tokens,
                  ws, logprob=None, status=None, stream=None):
    """:func:`greedy_accept` with drawn tokens: ``target`` [N] is drawn from
    each node's logits as by :func:`sample_tokens`, and the walk follows the
    children whose ``tokens`` are their parents' targets."""
    args, index = _sample_args(logits, uniform, sampling, target)
    n = args[0]
    for t, name in ((parent, "parent"), (tokens, "tokens"), (accept_len, "accept_len"),
                    (path, "path"), (out_tokens, "out_tokens"), (ws, "workspace")):
        if t is None:
            raise DfvError(f"{name} is required")
    _check(lib().dfv_sample_accept(
        *args, _ptr(parent, "parent", torch.int32, n, index),
        _ptr(tokens, "tokens", torch.int32, n, index),
        _ptr(target, "target", torch.int32, n, index),
        _ptr(logprob, "logprob", torch.float32, n, index),
        _ptr(accept_len, "accept_len", torch.int32, 1, index),
        _ptr(path, "path", torch.int32, n, index),
        _ptr(out_tokens, "out_tokens", torch.int32, n, index),
        _ptr(ws, "workspace", torch.uint8, 0, index), ws.numel(),
        _ptr(status, "status", torch.int32, 1, index), _stream(stream, index)),
        "dfv_sample_accept")


_PI = "3.1415926535897932384626433832795028841971693993751058209749445923078164062862090"


def _turns(base, rot_dim):
    """base ** (-2 i / rot_dim) / (2 pi) for i < rot_dim / 2, modulo 1, times 2^64,
    to the nearest integer (80 digits; doubles would be off by some hundred)."""
    if not base > 0:
        raise DfvError(f"base {base} must be positive")
    with decimal.localcontext(decimal.Context(prec=80)):
        # in units of 2^-192
        step = int(decimal.Decimal(base) ** (decimal.Decimal(-2) / rot_dim) * 2 ** 192)
        turn = int(2 ** 255 / decimal.Decimal(_PI))
    turns = []
    for _ in range(rot_dim // 2):
        turns.append((turn + (1 << 191) >> 192) % 2 ** 64)
        turn = turn * step >> 192
    return turns


class Rope:
    """Frequencies of the position rotation of :func:`qk_norm_rope`: the first
    ``rot_dim`` dims of a head (all by default) turn in pairs, pair i by
    ``base ** (-2 i / rot_dim)`` rad per position, or by ``inv_freq[i]``
    (rot_dim / 2 numbers). Pairs are dims (i, i + rot_dim / 2), or (2 i, 2 i + 1)
    with ``interleaved``. Kept as turns per position in 64-bit fractions: from
    ``base`` off by 2^-65, so angles are as exact at position 2^31 as at 1; from
    ``inv_freq``, which are doubles and divided as such, by 2^-52 of themselves."""

    def __init__(self, head_dim, rot_dim=None, base=10000.0, inv_freq=None, interleaved=False,
                 device="cuda"):
        rot_dim = head_dim if rot_dim is None else rot_dim
        if head_dim not in (64, 128, 256):
            raise DfvError(f"head_dim {head_dim} is not one of 64, 128, 256")
        if not 0 <= rot_dim <= head_dim or rot_dim % 16:
            raise DfvError(f"rot_dim {rot_dim} is not a multiple of 16 in [0, {head_dim}]")
        if inv_freq is None:
            turns = _turns(float(base), rot_dim) if rot_dim else []
        else:
            inv_freq = [float(f) for f in inv_freq]
            if len(inv_freq) != rot_dim // 2 or not all(math.isfinite(f) for f in inv_freq):
                raise DfvError(f"inv_freq must be {rot_dim // 2} finite numbers")
            turns = [int(math.fmod(f / (2.0 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64
                     for f in inv_freq]
        self.head_dim, self.rot_dim, self.interleaved = head_dim, rot_dim, bool(interleaved)
        self.turns = torch.tensor([t - (t >> 63 << 64) for t in turns], dtype=torch.int64,
                                  device=device)
        self._index, self._turns_ptr = self.turns.get_device(), self.turns.data_ptr()


def qk_norm_rope(q, k, v, rope, q_out, k_out, v_out=None, q_weight=None, k_weight=None, eps=1e-6,
                 positions=None, ctx_len=None, dropped=None, parent=None, status=None,
                 stream=None):
    """RMS norm of each head of ``q`` [N, Hq, D] and ``k`` [N, Hkv, D], times
    ``q_weight`` / ``k_weight`` (f32 [D]), then ``rope``'s rotation; ``v``
    [N, Hkv, D] (or None) is carried along. Sources are f32 or bf16 of any
    strides over contiguous heads (slices of one projection, say), outputs
    contiguous f32 or bf16, and may be the sources themselves. ``q`` or ``k``
    may be None. ``eps=None``: no norm.

    Row i stands at ``positions[i]`` (int32), or at ``ctx_len + dropped`` (both
    int32[1], ``dropped`` optional) plus its depth in the tree ``parent`` (int32
    [N], N <= MAX_NODES) or, without one, plus i."""
    first = q if q is not None else k
    if first is None:
        raise DfvError("q or k is required")
    if first.dim() != 3:
        raise DfvError("q and k must be [N, heads, D]")
    n, _, d = first.shape
    if rope.head_dim != d:
        raise DfvError(f"rope is for head_dim {rope.head_dim}, the rows have {d}")
    index = first.get_device()
    if index != torch._C._cuda_getDevice() or index != rope._index:
        _same_device(index, rope.turns)
    # one type for all sources, one for all outputs; a call of one token costs
    # little else than these checks, so they are written out
    src = first.dtype
    dst = (q_out if q is not None else k_out)
    if dst is None:
        raise DfvError("q_out is required" if q is not None else "k_out is required")
    dst = dst.dtype
    if src not in _ROWS or dst not in _ROWS:
        raise DfvError("sources and outputs must be CUDA f32 or bf16 tensors")
    hq = hkv = sq = sqh = sk = skh = sv = svh = 0
    pq = pk = pv = oq = ok = ov = None
    if q is not None:
        hq = q.shape[1]
        sq, sqh, one = q.stride()
        pq, oq = _row_pair(q, q_out, "q", (n, hq, d), one, src, dst, index)
    if k is not None:
        if k.dim() != 3:
            raise DfvError("q and k must be [N, heads, D]")
        hkv = k.shape[1]
        sk, skh, one = k.stride()
        pk, ok = _row_pair(k, k_out, "k", (n, hkv, d), one, src, dst, index)
    if v is not None:
        if k is None:
            raise DfvError("v without k")
        if v.dim() != 3:
            raise DfvError("v must be [N, heads, D]")
        sv, svh, one = v.stride()
        pv, ov = _row_pair(v, v_out, "v", (n, hkv, d), one, src, dst, index)
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise DfvError("q_weight or k_weight without a norm")
        eps = -1.0
    elif not eps >= 0:
        raise DfvError(f"eps {eps} must be 0 or more")
    if positions is not None:
        if ctx_len is not None or dropped is not None or parent is not None:
            raise DfvError("positions are given: no ctx_len, dropped or parent beside them")
    elif ctx_len is None:
        raise DfvError("ctx_len or positions are required")
    elif parent is not None and n > MAX_NODES:
        raise DfvError(f"{n} tree nodes, at most {MAX_NODES}")
    _check(lib().dfv_qk_norm_rope(
        n, hq, hkv, d, pq, pk, pv, DTYPE_F32 if src is torch.float32 else DTYPE_BF16, sq, sqh, sk,
        skh, sv, svh, _ptr(q_weight, "q_weight", torch.float32, d, index),
        _ptr(k_weight, "k_weight", torch.float32, d, index), eps,
        rope._turns_ptr, rope.rot_dim, rope.interleaved,
        _ptr(positions, "positions", torch.int32, n, index),
        _ptr(parent, "parent", torch.int32, n, index),
        _ptr(ctx_len, "ctx_len", torch.int32, 1, index),
        _ptr(dropped, "dropped", torch.int32, 1, index), oq, ok, ov,
        DTYPE_F32 if dst is torch.float32 else DTYPE_BF16,
        _ptr(status, "status", torch.int32, 1, index), _stream(stream, index)),
        "dfv_qk_norm_rope")


def _row_pair(x, out, name, shape, one, src, dst, index):
    """Addresses of rows [N, heads, D] and of the contiguous output for them."""
    if x.dtype is not src or x.get_device() != index:
        raise DfvError(f"{name} must be a {src} tensor on cuda:{index}")
    if x.shape != shape:
        raise DfvError(f"{name} has shape {tuple(x.shape)}, expected {shape}")
    if one != 1 and x.numel():
        raise DfvError(f"{name} rows must be contiguous")
    if (out is None or out.dtype is not dst or out.get_device() != index
            or not out.is_contiguous()):
        raise DfvError(f"{name}_out must be a contiguous {dst} tensor on cuda:{index}")
    if out.shape != shape:
        raise DfvError(f"{name}_out has shape {tuple(out.shape)}, expected {shape}")
    return x.data_ptr(), out.data_ptr()


def kv_commit(cache, accept_len, path, tree_k, tree_v, status=None, stream=None):
    n = tree_k.shape[0]
    _dev(tree_k, "tree_k", _BF16)
    _dev(tree_v, "tree_v", _BF16)
    _dev(accept_len, "accept_len", _I32, 1)
    _dev(path, "path", _I32)
    if isinstance(cache, Int8Cache):
        if tuple(tree_k.shape) != (n, cache.n_kv_heads, cache.head_dim) or \
                tree_v.shape != tree_k.shape:
            raise DfvError("tree_k and tree_v must be [N, Hkv, D] of the cache")
        _dev(path, "path", _I32, n)
        _same_device(cache._index, accept_len, path, tree_k, tree_v, status)
        _check(lib().dfv_kv8_commit(
            cache.handle, n, accept_len.data_ptr(), path.data_ptr(), tree_k.data_ptr(),
            tree_v.data_ptr(), cache._status_ptr if status is None else status.data_ptr(),
            _stream(stream)), "dfv_kv8_commit")
        return
    _check(lib().dfv_kv_commit(
        n, cache.n_kv_heads, cache.head_dim, cache.kv_format, cache.capacity, cache.ctx_len.data_ptr(),
        accept_len.data_ptr(), path.data_ptr(), tree_k.data_ptr(), tree_v.data_ptr(),
        cache.k.data_ptr(), cache.v.data_ptr(), _p(status), _stream(stream)), "dfv_kv_commit")


def _as_bf16(logits):
    """Logits given as bf16 bit patterns in int16, as bf16."""
    return logits if logits.dtype != torch.int16 else logits.view(torch.bfloat16)


class VerifyStep:
    """Outputs and workspace of the verify step for one problem shape; call
    :meth:`run` once per step. All buffers live on the device.

    ``pipelined=True`` launches each step so that it overlaps the previous
    kernel of the stream (``DFV_STEP_PIPELINED``); the object then keeps two
    workspaces and uses them in turn, as consecutive pipelined steps need.

    ``fmt="int8"`` plans for an :class:`Int8Cache`: the step is then the
    attention, the argmax with the walk, and the commit, launched one after
    the other (not pipelined, no ``tree_as_cache``).

    ``top=K`` also gives, per node, the log probability of its argmax token
    (``logprob``; the emitted tokens are the path's), the entropy of its
    logits (``entropy``) and its K most probable tokens (``top_ids``,
    ``top_logprobs``); ``top=0`` the first two alone.

    ``sampling`` (a :class:`Sampling`) draws each node's token instead of taking
    the argmax (:func:`sample_accept`; ``run`` then takes ``uniform``, N random
    numbers): ``argmax`` holds the drawn tokens, ``draw_logprob`` their log
    probabilities. The step is then attention, draw with walk, and commit,
    launched one after the other, over any cache (not pipelined)."""

    sampling = None

    def __init__(self, n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity, vocab,
                 max_depth=16, device="cuda", pipelined=False, fmt="q4_0", top=None,
                 sampling=None):
        if top is not None and not 0 <= top <= min(MAX_TOP, vocab):
            raise DfvError(f"top={top} alternatives, at most {min(MAX_TOP, vocab)}")
        self.shape = (n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity, vocab)
        self.max_depth = max_depth
        dev = torch.device(device)
        self.out = torch.empty(n_nodes, n_q_heads, head_dim, dtype=torch.float32, device=dev)
        self.lse = torch.empty(n_nodes, n_q_heads, dtype=torch.float32, device=dev)
        self.argmax = torch.empty(n_nodes, dtype=torch.int32, device=dev)
        self.accept_len = torch.zeros(1, dtype=torch.int32, device=dev)
        self.path = torch.empty(n_nodes, dtype=torch.int32, device=dev)
        self.out_tokens = torch.empty(n_nodes, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.int8 = fmt == "int8"
        if not self.int8:
            _fmt_code(fmt)
        elif pipelined:
            raise DfvError("pipelined is not available with an Int8Cache")
        self.sampling = sampling
        if sampling is not None:
            if pipelined:
                raise DfvError("pipelined is not available with sampling")
            if not isinstance(sampling, Sampling):
                raise DfvError("sampling must be a Sampling")
            self.draw_logprob = torch.empty(n_nodes, dtype=torch.float32, device=dev)
        if self.int8:
            nb = int8_attn_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window,
                                           capacity)
        elif sampling is not None:
            nb = attn_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity)
        else:
            nb = step_workspace_bytes(n_nodes, n_q_heads, n_kv_heads, head_dim, window, capacity,
                                      vocab)
        if nb == 0:
            raise DfvError(f"unsupported step shape {self.shape}")
        if sampling is not None:
            accept = sample_accept_workspace_bytes(n_nodes, vocab)
            if accept == 0:
                raise DfvError(f"unsupported step shape {self.shape}")
            self.accept_ws = workspace(accept, device=dev)
        elif self.int8:
            self.accept_ws = workspace(accept_workspace_bytes(n_nodes, vocab), device=dev)
        self.top = top
        if top is not None:
            self.logprob = torch.empty(n_nodes, dtype=torch.float32, device=dev)
            self.entropy = torch.empty(n_nodes, dtype=torch.float32, device=dev)
            self.top_ids = torch.empty(n_nodes, top, dtype=torch.int32, device=dev) if top else None
            self.top_logprobs = torch.empty(n_nodes, top, dtype=torch.float32,
                                            device=dev) if top else None
        self.pipelined = bool(pipelined)
        self.workspaces = [workspace(nb, device=dev) for _ in range(2 if self.pipelined else 1)]
        self.ws = self.workspaces[0]
        self._turn = 0

    def run(self, cache, q, tree_k, tree_v, parent, tokens, logits, scale=0.0, stream=None,
            tree_as_cache=False, uniform=None):
        n, hq, hkv, d, window, cap, vocab = self.shape
        if cache.capacity != cap:
            raise DfvError("cache capacity differs from the planned one")
        if isinstance(cache, Int8Cache) != self.int8:
            raise DfvError("the step is planned for another kind of cache")
        if (uniform is None) != (self.sampling is None):
            raise DfvError("uniform goes with a step planned with sampling, and only with one")
        if self.int8 or self.sampling is not None:
            for t, name, shape in ((q, "q", (n, hq, d)), (tree_k, "tree_k", (n, hkv, d)),
                                   (tree_v, "tree_v", (n, hkv, d)), (logits, "logits", (n, vocab))):
                if tuple(t.shape) != shape:
                    raise DfvError(f"{name} has shape {tuple(t.shape)}, the step is planned for "
                                   f"{shape}")
            _dev(parent, "parent", _I32, n)
            _dev(tokens, "tokens", _I32, n)
            _dev(logits, "logits", (torch.float32,) + _BF16)
            if self.sampling is not None:
                # before the first launch: what the draw would refuse
                _dev(uniform, "uniform", _F32, n)
                _same_device(logits.get_device(), uniform)
                self.sampling.check(n, logits.get_device())
            tree_verify_attn(cache, q, tree_k, tree_v, parent, window, self.max_depth, self.out,
                             self.lse, self.ws, scale=scale, status=self.status, stream=stream,
                             tree_as_cache=tree_as_cache)
            if self.sampling is not None:
                sample_accept(_as_bf16(logits), uniform, self.sampling, parent, tokens,
                              self.argmax, self.accept_len, self.path, self.out_tokens,
                              self.accept_ws, logprob=self.draw_logprob, status=self.status,
                              stream=stream)
            else:
                greedy_accept(logits, parent, tokens, self.argmax, self.accept_len, self.path,
                              self.out_tokens, self.accept_ws, status=self.status, stream=stream)
            kv_commit(cache, self.accept_len, self.path, tree_k, tree_v, status=self.status,
                      stream=stream)
            self._logprobs(logits, stream)
            return
        _dev(q, "q", _BF16, n * hq * d)
        _dev(tree_k, "tree_k", _BF16, n * hkv * d)
        _dev(tree_v, "tree_v", _BF16, n * hkv * d)
        _dev(parent, "parent", _I32, n)
        _dev(tokens, "tokens", _I32, n)
        _dev(logits, "logits", (torch.float32,) + _BF16, n * vocab)
        dt = DTYPE_F32 if logits.dtype == torch.float32 else DTYPE_BF16
        kvf = (cache.kv_format | (KV_TREE_AS_CACHE if tree_as_cache else 0)
               | (STEP_PIPELINED if self.pipelined else 0))
        ws = self.workspaces[self._turn]
        self._turn = (self._turn + 1) % len(self.workspaces)
        _check(lib().dfv_verify_step(
            n, self.max_depth, hq, hkv, d, window, kvf, cap, vocab, dt,
            cache.ctx_len.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), q.data_ptr(),
            tree_k.data_ptr(), tree_v.data_ptr(), parent.data_ptr(), tokens.data_ptr(),
            logits.data_ptr(), float(scale), self.out.data_ptr(), self.lse.data_ptr(),
            self.argmax.data_ptr(), self.accept_len.data_ptr(), self.path.data_ptr(),
            self.out_tokens.data_ptr(), ws.data_ptr(), ws.numel(),
            self.status.data_ptr(), _stream(stream)), "dfv_verify_step")
        self._logprobs(logits, stream)

    def _logprobs(self, logits, stream):
        if self.top is None:
            return
        # a step takes any shape of n * vocab logits
        n, vocab = self.shape[0], self.shape[-1]
        logits = logits.view(-1)[:n * vocab].view(n, vocab)
        token_logprobs(_as_bf16(logits), self.argmax, self.logprob, self.entropy, self.top_ids,
                       self.top_logprobs, status=self.status, stream=stream)
