"""Key/value cache: binding of ``include/sdpa_cache.h``.

``KVCache`` names the tensors of a cache; ``cache_forward``, ``cache_append``,
``cache_weigh`` and ``cache_evict`` are the calls a PyTorch user makes, each
over the C entry point of the same name. All work runs in the CUDA library on
torch's current stream; the calls can be captured into a CUDA graph. They serve
decoding: none of them records a gradient.

A decoding step of a model that drafts tokens:

    o, lse = cache_forward(cache, q, k, v, scale=s, tree=masks)  # draft rows
    ...                                       # the caller verifies the drafts
    cache_append(cache, k, v, index=accepted, counts=n_accepted)
    cache_weigh(cache, q, lse, scale=s, q_pos=accepted_positions)
    cache_evict(cache, budget, first=4, recent=256)
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

_i64x3 = ctypes.c_int64 * 3
_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class SdpaCache(ctypes.Structure):
    """Mirror of ``sdpa_cache`` (field order and types as in the header)."""
    _fields_ = [
        ("dtype", _i32), ("reserved0", _i32),
        ("b", _i64), ("h_kv", _i64), ("d", _i64),
        ("n_pages", _i64), ("page_size", _i64), ("max_pages", _i64),
        ("k", _vp), ("v", _vp), ("k_stride", _i64x3), ("v_stride", _i64x3),
        ("page_table", _vp), ("lengths", _vp), ("next_pos", _vp), ("positions", _vp),
        ("weights", _vp), ("status", _vp),
    ]


class SdpaCacheFwdParams(ctypes.Structure):
    _fields_ = [
        ("s_q", _i64), ("h_q", _i64), ("window_left", _i64),
        ("scale", ctypes.c_float), ("reserved0", _i32),
        ("q", _vp), ("k", _vp), ("v", _vp),
        ("q_stride", _i64x3), ("k_stride", _i64x3), ("v_stride", _i64x3), ("o_stride", _i64x3),
        ("tree", _vp), ("seq_q_lens", _vp), ("sink", _vp), ("o", _vp), ("lse", _vp),
    ]


class SdpaCacheAppendParams(ctypes.Structure):
    _fields_ = [
        ("layout", _i32), ("reserved0", _i32), ("s", _i64), ("n", _i64), ("total", _i64),
        ("k", _vp), ("v", _vp), ("k_stride", _i64x3), ("v_stride", _i64x3),
        ("index", _vp), ("counts", _vp), ("offsets", _vp),
    ]


class SdpaCacheWeighParams(ctypes.Structure):
    _fields_ = [
        ("s_q", _i64), ("h_q", _i64), ("window_left", _i64),
        ("scale", ctypes.c_float), ("reserved0", _i32),
        ("q", _vp), ("q_stride", _i64x3), ("lse", _vp), ("q_pos", _vp),
    ]


class SdpaCacheEvictParams(ctypes.Structure):
    _fields_ = [("keep", _i64), ("first", _i64), ("recent", _i64)]


ENTRY_POINTS = ("sdpa_cache_bytes", "sdpa_cache_fwd_params_bytes", "sdpa_cache_append_params_bytes",
                "sdpa_cache_weigh_params_bytes", "sdpa_cache_evict_params_bytes",
                "sdpa_cache_fwd_workspace_bytes", "sdpa_cache_fwd", "sdpa_cache_append",
                "sdpa_cache_weigh", "sdpa_cache_evict_workspace_bytes", "sdpa_cache_evict",
                "sdpa_cache_check_status", "sdpa_cache_test_hook")


def bind(lib) -> None:
    """Argument and result types of the cache's entry points."""
    C, sz, st = ctypes.POINTER(SdpaCache), ctypes.c_size_t, ctypes.c_int
    for name in ENTRY_POINTS[:5]:
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = sz
    for name, params in (("fwd", SdpaCacheFwdParams), ("evict", SdpaCacheEvictParams)):
        f = getattr(lib, f"sdpa_cache_{name}_workspace_bytes")
        f.argtypes, f.restype = [C, ctypes.POINTER(params)], sz
        f = getattr(lib, f"sdpa_cache_{name}")
        f.argtypes, f.restype = [C, ctypes.POINTER(params), _vp, sz, _vp], st
    for name, params in (("append", SdpaCacheAppendParams), ("weigh", SdpaCacheWeighParams)):
        f = getattr(lib, f"sdpa_cache_{name}")
        f.argtypes, f.restype = [C, ctypes.POINTER(params), _vp], st
    lib.sdpa_cache_check_status.argtypes, lib.sdpa_cache_check_status.restype = [C, _vp], st
    lib.sdpa_cache_test_hook.argtypes, lib.sdpa_cache_test_hook.restype = [_i64, _i32], st


def _lib():
    from . import load
    return load()


def _check(code: int, where: str) -> None:
    if code:
        from . import SdpaError, last_error
        raise SdpaError(code, where, last_error())


class _Calls:
    """The entry points with their parameter blocks as packed bytes (the layout
    of the structs above), and torch's current stream: filling a ctypes
    structure field by field costs more than the smallest call's kernel."""

    def __init__(self):
        import torch
        lib = _lib()
        for name in ("fwd", "evict"):
            f = lib[f"sdpa_cache_{name}"]
            f.argtypes, f.restype = [_vp, ctypes.c_char_p, _vp, ctypes.c_size_t, _vp], ctypes.c_int
            setattr(self, name, f)
        for name in ("append", "weigh"):
            f = lib[f"sdpa_cache_{name}"]
            f.argtypes, f.restype = [_vp, ctypes.c_char_p, _vp], ctypes.c_int
            setattr(self, name, f)
        self.empty, self.float32, self.int32, self.int64, self.uint8 = (
            torch.empty, torch.float32, torch.int32, torch.int64, torch.uint8)
        self.stream = torch._C._cuda_getCurrentRawStream


_FWD = struct.Struct("3qfi3Q12q5Q")
_APPEND = struct.Struct("2i3q2Q6q3Q")
_WEIGH = struct.Struct("3qfiQ3q2Q")
_EVICT = struct.Struct("3q")
_calls = None


def _c() -> _Calls:
    global _calls
    if _calls is None:
        _calls = _Calls()
    return _calls


# ----------------------------------------------------- one-to-one C entry points

def sdpa_cache_fwd_workspace_bytes(cache: SdpaCache, params: SdpaCacheFwdParams) -> int:
    return int(_lib().sdpa_cache_fwd_workspace_bytes(cache, params))


def sdpa_cache_fwd(cache, params, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().sdpa_cache_fwd(cache, params, workspace, workspace_bytes, stream)


def sdpa_cache_append(cache, params, stream: int) -> int:
    return _lib().sdpa_cache_append(cache, params, stream)


def sdpa_cache_weigh(cache, params, stream: int) -> int:
    return _lib().sdpa_cache_weigh(cache, params, stream)


def sdpa_cache_evict_workspace_bytes(cache: SdpaCache, params: SdpaCacheEvictParams) -> int:
    return int(_lib().sdpa_cache_evict_workspace_bytes(cache, params))


def sdpa_cache_evict(cache, params, workspace: int, workspace_bytes: int, stream: int) -> int:
    return _lib().sdpa_cache_evict(cache, params, workspace, workspace_bytes, stream)


def sdpa_cache_check_status(cache, stream: int) -> int:
    return _lib().sdpa_cache_check_status(cache, stream)


def sdpa_cache_test_hook(wait_limit_ns: int, flags: int) -> int:
    """Test-only: device wait limit, and copies left out so that waits run out,
    for this thread's later cache calls ((0, 0) restores normal operation)."""
    return _lib().sdpa_cache_test_hook(wait_limit_ns, flags)


# ------------------------------------------------------------- torch helpers

def _wrong(name, t, shape, device, dtype):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    raise ValueError(f"{name}: expected device {device}, got {t.device}")


def _strides(name, t, shape, device, dtype):
    """Element strides of all but the feature dimension of a tensor of this
    shape; 0 where the dimension has no second entry to address."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _wrong(name, t, shape, device, dtype)
    st = t.stride()
    if st[-1] != 1:
        raise ValueError(f"{name}: the feature dimension must be contiguous (stride 1)")
    return [s if n > 1 else 0 for s, n in zip(st[:-1], shape)]


def _strides4(name, t, shape, device, dtype):
    """The same of a call's tensor [.., .., .., d]: any stride serves where
    there is no second entry, as long as the library's check takes it."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _wrong(name, t, shape, device, dtype)
    x, y, z, feature = t.stride()
    if feature != 1 or (x | y | z) & 7:
        return _strides(name, t, shape, device, dtype)
    return x, y, z


def _flat(name, t, shape, device, dtype):
    """Address of a contiguous array of this shape and type; 0 for None."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _wrong(name, t, shape, device, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _apart(name, t):
    """An output's rows must not share memory (an expanded dimension)."""
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError(f"{name}: rows share memory (an expanded tensor)")


class KVCache:
    """The tensors of a paged key/value cache (see include/sdpa_cache.h).

    k, v: [n_pages, page_size, h_kv, d] bf16/f16; lengths: int32 [b];
    page_table: int32 [b, max_pages] (without it page i is sequence i's only
    one); next_pos: int32 [b] and positions: int32 [b, h_kv, capacity], both or
    neither; weights: fp32 [b, h_kv, capacity]. All on one CUDA device, and
    changed in place by the calls. `status` is the int32 word that holds the
    first problem found on the device (see check_status).
    """

    def __init__(self, k, v, lengths, *, page_table=None, next_pos=None, positions=None, weights=None):
        import torch
        from . import SDPA_BF16, SDPA_F16
        if k.dim() != 4:
            raise ValueError(f"k: expected [n_pages, page_size, h_kv, d], got {tuple(k.shape)}")
        if k.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"unsupported dtype {k.dtype}")
        n_pages, page_size, h_kv, d = k.shape
        dev, b = k.device, lengths.numel()
        i32 = torch.int32
        c = SdpaCache()
        c.dtype = SDPA_BF16 if k.dtype == torch.bfloat16 else SDPA_F16
        c.b, c.h_kv, c.d, c.n_pages, c.page_size = b, h_kv, d, n_pages, page_size
        c.k_stride = _i64x3(*_strides("k", k, tuple(k.shape), dev, k.dtype))
        c.v_stride = _i64x3(*_strides("v", v, tuple(k.shape), dev, k.dtype))
        _apart("k", k)
        _apart("v", v)
        if page_table is not None:
            if page_table.dim() != 2:
                raise ValueError("page_table: expected [b, max_pages]")
            c.max_pages = page_table.shape[1]
            c.page_table = _flat("page_table", page_table, (b, page_table.shape[1]), dev, i32)
        else:
            c.max_pages = 1
            if n_pages < b:
                raise ValueError(f"without a page_table each sequence needs a page: {n_pages} pages, {b} sequences")
        self.capacity = int(c.max_pages * page_size)
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.lengths = _flat("lengths", lengths, (b,), dev, i32)
        c.next_pos = _flat("next_pos", next_pos, (b,), dev, i32)
        c.positions = _flat("positions", positions, (b, h_kv, self.capacity), dev, i32)
        c.weights = _flat("weights", weights, (b, h_kv, self.capacity), dev, torch.float32)
        if (positions is None) != (next_pos is None):
            raise ValueError("positions and next_pos: both or neither")
        self.status = torch.zeros(1, dtype=i32, device=dev)
        c.status = self.status.data_ptr()
        self.k, self.v, self.lengths, self.page_table = k, v, lengths, page_table
        self.next_pos, self.positions, self.weights = next_pos, positions, weights
        self.b, self.h_kv, self.d, self.dtype, self.device = b, h_kv, d, k.dtype, dev
        self.params = c
        self._ref, self._key, self._index = ctypes.addressof(c), (b, h_kv, d, dev, k.dtype), dev.index or 0
        self._ws_bytes = {}     # workspace bytes of the calls made so far, by their sizes

    _own = frozenset(("k", "v", "lengths", "page_table", "next_pos", "positions", "weights", "status", "params", "capacity",
                      "b", "h_kv", "d", "dtype", "device"))

    def __setattr__(self, name, value):
        # the calls use the addresses taken by the constructor: another tensor under the name would not be seen
        if name in self._own and "_ws_bytes" in self.__dict__:
            raise AttributeError(f"{name}: a cache's tensors are changed in place (or make another KVCache)")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, b: int, h_kv: int, d: int, max_len: int, *, dtype, device, page_size: int = 64,
              track: bool = False) -> "KVCache":
        """An empty cache with room for max_len keys in each of b sequences;
        `track`: with positions and weights, as weighing and eviction need."""
        import torch
        per = -(-max_len // page_size)
        kw = dict(dtype=torch.int32, device=device)
        k, v = (torch.zeros(b * per, page_size, h_kv, d, dtype=dtype, device=device) for _ in range(2))
        extra = {}
        if track:
            extra = dict(next_pos=torch.zeros(b, **kw), positions=torch.full((b, h_kv, per * page_size), -1, **kw),
                         weights=torch.zeros(b, h_kv, per * page_size, device=device))
        return cls(k, v, torch.zeros(b, **kw), page_table=torch.arange(b * per, **kw).view(b, per), **extra)

    def check_status(self) -> None:
        """Synchronises torch's current stream and raises if a call found a
        problem on the device (a length, count, index or page out of range);
        clears it."""
        import torch
        _check(sdpa_cache_check_status(self.params, torch.cuda.current_stream(self.device).cuda_stream),
               "sdpa_cache_check_status")


def _ws_size(cache, key, size, params, p):
    """Workspace bytes of a call, kept by `key`, the arguments they depend on."""
    n = size(cache.params, params.from_buffer_copy(p))
    if n == 0:
        from . import SDPA_ERR_INVALID_ARG, SdpaError, last_error
        if last_error():
            raise SdpaError(SDPA_ERR_INVALID_ARG, size.__name__, last_error())
    if len(cache._ws_bytes) >= 256:
        cache._ws_bytes.clear()
    cache._ws_bytes[key] = n
    return n


def _given(workspace, c):
    """Bytes of the caller's workspace."""
    if workspace.dtype is not c.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor")
    return workspace.numel()


def cache_forward(cache: KVCache, q, k, v, *, scale: float, window_left: int = -1, tree=None, seq_q_lens=None,
                  sink=None, out=None, lse=None, workspace=None, check_status: bool = False):
    """O and LSE of up to 64 new tokens per sequence over the cached keys and
    over each other.

    q: [b, s_q, h_q, d], k, v: [b, s_q, h_kv, d] of the new tokens (not in the
    cache yet); tree: int64 [b, s_q], bit u of tree[i, r] set for r itself and
    each token u that r descends from (0: a padding row; None: a chain);
    seq_q_lens: int32 [b] real rows of each sequence; sink: fp32 [h_q].
    Returns (o, lse) with o like q and lse fp32 [b, h_q, s_q]. Tensors that
    require a gradient are taken, and nothing is recorded for one.
    """
    c = _calls or _c()
    if q.dim() != 4:
        raise ValueError(f"q: expected [b, s_q, h_q, d], got {tuple(q.shape)}")
    _, s_q, h_q, _ = q.shape
    b, h_kv, d, dev, dt = cache._key
    rows, kv = (b, s_q, h_q, d), (b, s_q, h_kv, d)
    sq = _strides4("q", q, rows, dev, dt)
    sk = _strides4("k", k, kv, dev, dt)
    sv = _strides4("v", v, kv, dev, dt)
    if out is None:
        out = c.empty(rows, dtype=dt, device=dev)
        so = (s_q * h_q * d, h_q * d, d)
    else:
        _apart("out", out)
        so = _strides("out", out, rows, dev, dt)
    if lse is None:
        lse = c.empty((b, h_q, s_q), dtype=c.float32, device=dev)
        lse_at = lse.data_ptr()
    else:
        lse_at = _flat("lse", lse, (b, h_q, s_q), dev, c.float32)
    p = _FWD.pack(s_q, h_q, window_left, scale, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), *sq, *sk, *sv, *so,
                  0 if tree is None else _flat("tree", tree, (b, s_q), dev, c.int64),
                  0 if seq_q_lens is None else _flat("seq_q_lens", seq_q_lens, (b,), dev, c.int32),
                  0 if sink is None else _flat("sink", sink, (h_q,), dev, c.float32), out.data_ptr(), lse_at)
    if workspace is None:
        key = s_q, h_q, window_left
        n = cache._ws_bytes.get(key)
        if n is None:
            n = _ws_size(cache, key, sdpa_cache_fwd_workspace_bytes, SdpaCacheFwdParams, p)
        if n:
            workspace = c.empty(n, dtype=c.uint8, device=dev)
    else:
        n = _given(workspace, c)
    code = c.fwd(cache._ref, p, workspace.data_ptr() if n else 0, n, c.stream(cache._index))
    if code:
        _check(code, "sdpa_cache_fwd")
    if check_status:
        cache.check_status()
    return out, lse


def cache_append(cache: KVCache, k, v, *, index=None, counts=None, offsets=None, max_seqlen: Optional[int] = None,
                 check_status: bool = False) -> None:
    """Puts new keys and values behind each sequence's cached ones.

    k, v: [b, s, h_kv, d], of which sequence i appends its first counts[i] rows
    (int32 [b]; all of them without counts), or rows index[i, 0],
    index[i, 1], .. (int32 [b, n]) where an index is given; or packed,
    [total, h_kv, d] with offsets (int32 [b + 1]) and max_seqlen, the most rows
    of a sequence.
    """
    c = _calls or _c()
    b, h_kv, d, dev, dt = cache._key
    n = total = 0
    if k.dim() == 3:
        if offsets is None or max_seqlen is None:
            raise ValueError("packed k, v need offsets and max_seqlen")
        if index is not None:
            raise ValueError("index: only with k, v of [b, s, h_kv, d]")
        layout, s, total = 1, max_seqlen, k.shape[0]
        shape = (total, h_kv, d)
        sk, sv = (0, *_strides("k", k, shape, dev, dt)), (0, *_strides("v", v, shape, dev, dt))
    else:
        if offsets is not None:
            raise ValueError("offsets: only with packed k, v ([total, h_kv, d])")
        if k.dim() != 4:
            raise ValueError(f"k: expected [b, s, h_kv, d] or [total, h_kv, d], got {tuple(k.shape)}")
        layout, s = 0, k.shape[1]
        shape = (b, s, h_kv, d)
        sk, sv = _strides4("k", k, shape, dev, dt), _strides4("v", v, shape, dev, dt)
    if index is not None:
        if index.dim() != 2:
            raise ValueError("index: expected [b, n]")
        n = index.shape[1]
        if n == 0:
            s = 0       # no row of any sequence (and no address of an empty index)
    p = _APPEND.pack(layout, 0, s, n, total, k.data_ptr(), v.data_ptr(), *sk, *sv,
                     0 if index is None else _flat("index", index, (b, n), dev, c.int32),
                     0 if counts is None else _flat("counts", counts, (b,), dev, c.int32),
                     0 if offsets is None else _flat("offsets", offsets, (b + 1,), dev, c.int32))
    _check(c.append(cache._ref, p, c.stream(cache._index)), "sdpa_cache_append")
    if check_status:
        cache.check_status()


def cache_weigh(cache: KVCache, q, lse, *, scale: float, window_left: int = -1, q_pos=None,
                check_status: bool = False) -> None:
    """Adds to each cached key's weight the attention it gets from given rows.

    q: [b, s_q, h_q, d] and lse: fp32 [b, h_q, s_q], as cache_forward or
    forward took and gave them; q_pos: int32 [b, s_q] positions of the rows
    (negative: the row does not count), or None for the last s_q tokens.
    """
    c = _calls or _c()
    if q.dim() != 4:
        raise ValueError(f"q: expected [b, s_q, h_q, d], got {tuple(q.shape)}")
    _, s_q, h_q, _ = q.shape
    b, _, d, dev, dt = cache._key
    p = _WEIGH.pack(s_q, h_q, window_left, scale, 0, q.data_ptr(), *_strides4("q", q, (b, s_q, h_q, d), dev, dt),
                    _flat("lse", lse, (b, h_q, s_q), dev, c.float32),
                    0 if q_pos is None else _flat("q_pos", q_pos, (b, s_q), dev, c.int32))
    _check(c.weigh(cache._ref, p, c.stream(cache._index)), "sdpa_cache_weigh")
    if check_status:
        cache.check_status()


def cache_evict(cache: KVCache, keep: int, *, first: int = 0, recent: int = 0, workspace=None,
                check_status: bool = False) -> None:
    """Brings each sequence that holds more than `keep` keys back to `keep`:
    the keys at positions below `first`, the `recent` last positions and the
    heaviest of the others stay, for each kv-head on its own."""
    c = _calls or _c()
    p = _EVICT.pack(keep, first, recent)
    if workspace is None:
        key = "evict", keep, first, recent
        n = cache._ws_bytes.get(key)
        if n is None:
            n = _ws_size(cache, key, sdpa_cache_evict_workspace_bytes, SdpaCacheEvictParams, p)
        if n:
            workspace = c.empty(n, dtype=c.uint8, device=cache.device)
    else:
        n = _given(workspace, c)
    _check(c.evict(cache._ref, p, workspace.data_ptr() if n else 0, n, c.stream(cache._index)), "sdpa_cache_evict")
    if check_status:
        cache.check_status()
