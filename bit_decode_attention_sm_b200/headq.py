"""Python binding of libheadq (``include/headq.h``): argument marshalling only.

Every computation runs in the CUDA kernels of ``libheadq.so``; this module
only allocates device memory through PyTorch, passes pointers, sizes and the
current CUDA stream, and turns status codes into exceptions.  There is no CPU
fallback: without the built library, or with tensors that are not on a CUDA
device, every call raises.

Names follow the C ABI: :func:`headq_calibrate`, :func:`headq_cache_write`,
:func:`headq_decode_attn`, :func:`headq_attn_kl`, the packed-batch calls
:func:`headq_cache_write_ragged`, :func:`headq_cache_read` and
:func:`headq_tree_attn`, plus :class:`HeadQCache` which owns the packed cache
planes.
"""

import contextlib
import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libheadq.so")

HEADQ_F32, HEADQ_BF16 = 0, 1
HEADQ_V_DENSE, HEADQ_V_2BIT = 0, 1
STATUS = {0: "HEADQ_OK", 1: "HEADQ_ERR_INVALID_ARG", 2: "HEADQ_ERR_UNSUPPORTED",
          3: "HEADQ_ERR_WORKSPACE", 4: "HEADQ_ERR_CUDA", 5: "HEADQ_ERR_DEVICE"}

# Every entry point declared in include/headq.h.
EXPORTS = ("headq_version", "headq_status_string", "headq_calibrate",
           "headq_calibrate_workspace_bytes", "headq_cache_write", "headq_decode_attn",
           "headq_decode_workspace_bytes", "headq_decode_plan", "headq_attn_kl",
           "headq_attn_kl_workspace_bytes", "headq_workspace_status",
           "headq_decode_attn_noalloc", "headq_decode_noalloc_status",
           "headq_decode_append", "headq_shard_seq_lens",
           "headq_merge_partials", "headq_a2_workspace_bytes", "headq_a2_scores",
           "headq_a2_select", "headq_a2_value_fixup", "headq_cache_write_ragged",
           "headq_cache_read", "headq_tree_attn", "headq_tree_workspace_bytes")


KMODES = {"token": 0, "channel": 1}  # headq_kmode


class HeadQError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s" % (fn, STATUS.get(status, status)))


class CacheStruct(ctypes.Structure):
    """Mirror of ``headq_cache``."""
    _fields_ = [("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("T_cap", ctypes.c_int),
                ("d", ctypes.c_int), ("r", ctypes.c_int), ("vmode", ctypes.c_int),
                ("v_dtype", ctypes.c_int),
                ("k_codes", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("k_min", ctypes.c_void_p), ("z_codes", ctypes.c_void_p),
                ("z_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("v_min", ctypes.c_void_p),
                ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("block_table", ctypes.c_void_p),
                ("kmode", ctypes.c_int)]


class SpanStruct(ctypes.Structure):
    """Mirror of ``headq_span``."""
    _fields_ = [("seq_lens", ctypes.c_void_p), ("cu", ctypes.c_void_p), ("T", ctypes.c_int),
                ("n", ctypes.c_int), ("rows", ctypes.c_int)]


class RowsStruct(ctypes.Structure):
    """Mirror of ``headq_rows``."""
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


_lib = None


def lib():
    """The loaded libheadq; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libheadq.so is not built: run "
                               "`python -m bit_decode_attention_sm_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        F = ctypes.c_float
        CP, SP, RP = (ctypes.POINTER(c) for c in (CacheStruct, SpanStruct, RowsStruct))
        sig = {
            "headq_version": ([], I),
            "headq_status_string": ([I], ctypes.c_char_p),
            "headq_calibrate": ([P, I, I, I, I, I, I, I, P, P, P, Z, P], I),
            "headq_calibrate_workspace_bytes": ([I, I, I, I], Z),
            "headq_cache_write": ([CP, P, P, I, I, I, P, P], I),
            "headq_decode_attn": ([CP, P, I, I, P, I, P, F, I, P, P, P, Z, P], I),
            "headq_decode_workspace_bytes": ([CP, I, I], Z),
            "headq_decode_plan": ([CP, I, I, P, P, P], I),
            "headq_attn_kl": ([CP, P, I, I, P, I, P, P, I, P, F, I, P, P, P, P, P, Z, P], I),
            "headq_attn_kl_workspace_bytes": ([CP, I, I], Z),
            "headq_workspace_status": ([P, P], I),
            "headq_decode_attn_noalloc": ([CP, P, I, I, P, I, P, F, I, P, P, P], I),
            "headq_decode_noalloc_status": ([P], I),
            "headq_decode_append": ([CP, P, P, I, P, I, I, P, I, P, F, I, P, P, P, Z, P], I),
            "headq_shard_seq_lens": ([P, I, I, I, I, P, P], I),
            "headq_merge_partials": ([P, P, I, I, I, Z, P, P, P], I),
            "headq_a2_workspace_bytes": ([CP, I, I, I], Z),
            "headq_a2_scores": ([CP, P, I, I, I, P, I, P, P, I, F, P, P, Z, P], I),
            "headq_a2_select": ([P, I, I, P, I, I, P, I, I, P, P, P], I),
            "headq_a2_value_fixup": ([CP, P, I, I, P, I, P, F, I, P, P, I, I, P, P, P], I),
            "headq_cache_write_ragged": ([CP, RP, RP, I, P, SP, P, P], I),
            "headq_cache_read": ([CP, SP, P, I, RP, RP, P, P], I),
            "headq_tree_attn": ([CP, RP, I, P, ctypes.c_longlong, SP, P, F, I, RP, P, P, Z, P], I),
            "headq_tree_workspace_bytes": ([CP, I, I, I], Z),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(fn, st):
    if st != 0:
        raise HeadQError(fn, st)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return HEADQ_F32
    if t.dtype == torch.bfloat16:
        return HEADQ_BF16
    raise TypeError("HeadQ tensors are float32 or bfloat16, got %s" % t.dtype)


def _cuda(t, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class HeadQCache:
    """Caller-owned packed HeadQ cache planes on one CUDA device.

    Planes follow ``headq_cache`` in include/headq.h: k_codes u8
    [B,Hkv,T_cap,d/4], k_scale/k_min f32 [B,Hkv,T_cap,NG], z_codes u8
    [B,Hkv,T_cap,r/2], z_scale f32 [B,Hkv,T_cap], and either v
    [B,Hkv,T_cap,d] (dense) or v_codes/v_scale/v_min (2-bit).
    """

    page_size = num_pages = max_pages = 0
    block_table = None
    kmode = "token"

    def __init__(self, B, Hkv, T_cap, d, r, vmode="dense", v_dtype=torch.bfloat16,
                 device="cuda", kmode="token"):
        if T_cap % (64 if kmode == "channel" else 16):
            raise ValueError("T_cap must be a multiple of 16 (64 for per-channel keys)")
        self.B, self.Hkv, self.T_cap, self.d, self.r = B, Hkv, T_cap, d, r
        self._alloc((B, Hkv, T_cap), vmode, v_dtype, device, kmode)

    def _alloc(self, lead, vmode, v_dtype, device, kmode="token"):
        d, r = self.d, self.r
        if kmode not in KMODES:
            raise ValueError("kmode is 'token' or 'channel'")
        self.vmode = vmode
        self.v_dtype = v_dtype
        self.kmode = kmode
        ng = d // min(32, d)
        u8, f32 = torch.uint8, torch.float32
        self.k_codes = torch.zeros(lead + (d // 4,), dtype=u8, device=device)
        # per-token groups, or (per-channel code) one row of d per 64-token block
        sshape = lead + (ng,) if kmode == "token" else lead[:-1] + (lead[-1] // 64, d)
        self.k_scale = torch.zeros(sshape, dtype=f32, device=device)
        self.k_min = torch.zeros(sshape, dtype=f32, device=device)
        self.z_codes = torch.zeros(lead + (max(r // 2, 1),), dtype=u8, device=device)
        self.z_scale = torch.zeros(lead, dtype=f32, device=device)
        self.v = self.v_codes = self.v_scale = self.v_min = None
        if vmode == "dense":
            self.v = torch.zeros(lead + (d,), dtype=v_dtype, device=device)
        elif vmode == "2bit":
            self.v_codes = torch.zeros(lead + (d // 4,), dtype=u8, device=device)
            self.v_scale = torch.zeros(lead + (ng,), dtype=f32, device=device)
            self.v_min = torch.zeros(lead + (ng,), dtype=f32, device=device)
        else:
            raise ValueError("vmode is 'dense' or '2bit'")

    @staticmethod
    def from_planes(k_codes, k_scale, k_min, z_codes=None, z_scale=None, v=None, v_codes=None,
                    v_scale=None, v_min=None, kmode="token", block_table=None):
        """A cache over planes that are allocated already (a server's pools): contiguous
        CUDA tensors laid out as the class says, nothing copied.  With ``block_table``
        (int32 [B, max_pages]) the planes are pools of pages and the result is a
        :class:`PagedHeadQCache`.  z_codes/z_scale None: rank 0."""
        lead, d = tuple(k_codes.shape[:3]), k_codes.shape[3] * 4
        r = 0 if z_codes is None else z_codes.shape[3] * 2
        ng = d // min(32, d)
        if kmode not in KMODES:
            raise ValueError("kmode is 'token' or 'channel'")
        if (v is None) == (v_codes is None):
            raise ValueError("either v (dense values) or v_codes, v_scale and v_min")
        u8, f32 = torch.uint8, torch.float32
        sshape = lead + (ng,) if kmode == "token" else lead[:2] + (lead[2] // 64, d)
        want = dict(k_codes=(k_codes, u8, lead + (d // 4,)), k_scale=(k_scale, f32, sshape),
                    k_min=(k_min, f32, sshape))
        if r:
            want.update(z_codes=(z_codes, u8, lead + (r // 2,)), z_scale=(z_scale, f32, lead))
        if v is None:
            want.update(v_codes=(v_codes, u8, lead + (d // 4,)), v_scale=(v_scale, f32, lead + (ng,)),
                        v_min=(v_min, f32, lead + (ng,)))
        else:
            _dtype_code(v)
            want.update(v=(v, v.dtype, lead + (d,)))
        for name, (t, dt, shape) in want.items():
            if _cuda(t, name) is None or t.dtype != dt or tuple(t.shape) != shape:
                raise ValueError("%s must be %s %s" % (name, dt, list(shape)))
            if t.device != k_codes.device:
                raise ValueError("%s is on %s, k_codes on %s" % (name, t.device, k_codes.device))
        if block_table is None:
            c = HeadQCache.__new__(HeadQCache)
            c.B, c.T_cap = lead[0], lead[2]
            if c.T_cap % (64 if kmode == "channel" else 16):
                raise ValueError("T_cap must be a multiple of 16 (64 for per-channel keys)")
        else:
            c = PagedHeadQCache.__new__(PagedHeadQCache)
            if _cuda(block_table, "block_table").dtype != torch.int32 or block_table.dim() != 2:
                raise ValueError("block_table must be int32 [B, max_pages]")
            c.B, c.max_pages = block_table.shape
            c.num_pages, c.page_size = lead[0], lead[2]
            if c.page_size <= 0 or c.page_size % 64:
                raise ValueError("page_size must be a positive multiple of 64")
            c.T_cap = c.max_pages * c.page_size
            c.block_table = block_table
        c.Hkv, c.d, c.r, c.kmode = lead[1], d, r, kmode
        c.vmode = "dense" if v_codes is None else "2bit"
        c.v_dtype = torch.bfloat16 if v is None else v.dtype
        c.k_codes, c.k_scale, c.k_min, c.z_codes, c.z_scale = k_codes, k_scale, k_min, z_codes, z_scale
        c.v, c.v_codes, c.v_scale, c.v_min = v, v_codes, v_scale, v_min
        if block_table is not None:
            c._table()
        return c

    def planes(self):
        out = dict(kc=self.k_codes, ks=self.k_scale, km=self.k_min, zc=self.z_codes,
                   zs=self.z_scale)
        if self.vmode == "2bit":
            out.update(vc=self.v_codes, vs=self.v_scale, vm=self.v_min)
        else:
            out.update(v=self.v)
        return out

    def nbytes_per_token(self):
        """Bytes one cached token of one KV head occupies in HBM."""
        ng = self.d // min(32, self.d)
        b = self.d // 4 + (8 * ng if self.kmode == "token" else self.d // 8) + self.r // 2 + 4
        if self.vmode == "2bit":
            b += self.d // 4 + 8 * ng
        else:
            b += self.d * (2 if self.v_dtype == torch.bfloat16 else 4)
        return b

    def _table(self):
        """The block table, as the kernels index it; it may have been assigned since the last call."""
        t = self.block_table
        if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_contiguous()
                or t.shape != (self.B, self.max_pages) or t.device != self.k_codes.device):
            raise ValueError("block_table must be contiguous int32 [%d, %d] on %s"
                             % (self.B, self.max_pages, self.k_codes.device))
        return t

    def struct(self):
        s = CacheStruct()
        s.B, s.Hkv, s.T_cap, s.d, s.r = self.B, self.Hkv, self.T_cap, self.d, self.r
        s.vmode = HEADQ_V_DENSE if self.vmode == "dense" else HEADQ_V_2BIT
        s.v_dtype = HEADQ_BF16 if self.v_dtype == torch.bfloat16 else HEADQ_F32
        s.k_codes = self.k_codes.data_ptr()
        s.k_scale = self.k_scale.data_ptr()
        s.k_min = self.k_min.data_ptr()
        if self.z_codes is not None:
            s.z_codes = self.z_codes.data_ptr()
            s.z_scale = self.z_scale.data_ptr()
        if self.vmode == "dense":
            s.v = self.v.data_ptr()
        else:
            s.v_codes = self.v_codes.data_ptr()
            s.v_scale = self.v_scale.data_ptr()
            s.v_min = self.v_min.data_ptr()
        if self.page_size:
            s.page_size, s.num_pages, s.max_pages = self.page_size, self.num_pages, self.max_pages
            s.block_table = self._table().data_ptr()
        s.kmode = KMODES[self.kmode]
        return s


class PagedHeadQCache(HeadQCache):
    """HeadQ cache planes held as pools of fixed-size pages (``headq_cache``
    paged layout): every plane is [num_pages, Hkv, page_size, ...] and
    ``block_table`` int32 [B, max_pages] names the pool page that holds tokens
    [i*page_size, (i+1)*page_size) of sequence b.  page_size is a multiple of
    64; a sequence holds up to T_cap = max_pages * page_size tokens.  The
    default block table gives sequence b pages b*max_pages .. b*max_pages +
    max_pages - 1 (it needs num_pages >= B * max_pages); any other table may be
    assigned to ``block_table`` before a call."""

    def __init__(self, B, Hkv, d, r, page_size, num_pages, max_pages, vmode="dense",
                 v_dtype=torch.bfloat16, device="cuda", block_table=None, kmode="token"):
        if page_size <= 0 or page_size % 64:
            raise ValueError("page_size must be a positive multiple of 64")
        self.B, self.Hkv, self.d, self.r = B, Hkv, d, r
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages
        self.T_cap = max_pages * page_size
        if block_table is None:
            if num_pages < B * max_pages:
                raise ValueError("the default block table needs B * max_pages pages")
            block_table = torch.arange(B * max_pages, dtype=torch.int32).view(B, max_pages)
        self.block_table = block_table.to(device=device, dtype=torch.int32).contiguous()
        if tuple(self.block_table.shape) != (B, max_pages):
            raise ValueError("block_table must be [B, max_pages]")
        self._alloc((num_pages, Hkv, page_size), vmode, v_dtype, device, kmode)


def headq_calibrate(q_cal, Hkv, r, center=False, stream=None):
    """Query-PCA basis per KV head: returns (U fp32 [Hkv,d,r], eig fp32 [Hkv,r])."""
    q_cal = _cuda(q_cal, "q_cal")
    N, Hq, d = q_cal.shape
    L = lib()
    U = torch.empty((Hkv, d, r), dtype=torch.float32, device=q_cal.device)
    eig = torch.empty((Hkv, r), dtype=torch.float32, device=q_cal.device)
    nws = L.headq_calibrate_workspace_bytes(N, Hq, Hkv, d)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device=q_cal.device)
    _check("headq_calibrate", L.headq_calibrate(
        _ptr(q_cal), _dtype_code(q_cal), N, Hq, Hkv, d, r, int(bool(center)), _ptr(U),
        _ptr(eig), _ptr(ws), nws, _stream(stream)))
    return U, eig


def headq_cache_write(cache, k, v, U, t0=0, stream=None):
    """Encode k (and store v) [B,Hkv,n,d] into cache positions [t0, t0+n)."""
    k = _cuda(k, "k")
    v = _cuda(v, "v")
    if v is not None and v.dtype != k.dtype:
        raise TypeError("k and v must have the same dtype")
    n = k.shape[2]
    U = _cuda(U, "U") if cache.r > 0 else None
    cs = cache.struct()
    _check("headq_cache_write", lib().headq_cache_write(
        ctypes.byref(cs), _ptr(k), _ptr(v), _dtype_code(k), int(t0), int(n), _ptr(U),
        _stream(stream)))


def decode_workspace(cache, Hq, T):
    """A zeroed device workspace sized for headq_decode_attn."""
    cs = cache.struct()
    n = lib().headq_decode_workspace_bytes(ctypes.byref(cs), Hq, T)
    return torch.zeros(n, dtype=torch.uint8, device=cache.k_codes.device)


def decode_plan(cache, Hq, T):
    """(splits, chunk, kernels per headq_decode_attn call, kernels per
    headq_decode_append call) for these sizes on the current device."""
    cs = cache.struct()
    sp, ch, ak = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    nk = lib().headq_decode_plan(ctypes.byref(cs), Hq, T, ctypes.byref(sp), ctypes.byref(ch),
                                 ctypes.byref(ak))
    return sp.value, ch.value, nk, ak.value


def attn_kl_workspace(cache, Hq, T):
    cs = cache.struct()
    n = lib().headq_attn_kl_workspace_bytes(ctypes.byref(cs), Hq, T)
    return torch.zeros(n, dtype=torch.uint8, device=cache.k_codes.device)


def headq_decode_attn(cache, q, U, T=None, seq_lens=None, sm_scale=None, corr_sign=1,
                      out=None, lse=None, ws=None, stream=None):
    """Decode attention over the cache; returns (out fp32 [B,Hq,d], lse fp32 [B,Hq])."""
    q = _cuda(q, "q")
    B, Hq, d = q.shape
    T = cache.T_cap if T is None else int(T)
    sm = 1.0 / math.sqrt(d) if sm_scale is None else float(sm_scale)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = decode_workspace(cache, Hq, T)
    seq_lens = _cuda(seq_lens, "seq_lens")
    U = _cuda(U, "U") if cache.r > 0 else None
    cs = cache.struct()
    _check("headq_decode_attn", lib().headq_decode_attn(
        ctypes.byref(cs), _ptr(q), _dtype_code(q), Hq, _ptr(seq_lens), T, _ptr(U), sm,
        int(corr_sign), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


def headq_decode_append(cache, k_new, v_new, q, U, T=None, seq_lens=None, sm_scale=None,
                        corr_sign=1, out=None, lse=None, ws=None, stream=None):
    """One decode step: write each sequence's new token (k_new, v_new [B,Hkv,d]) at
    position T_b - 1, then attend; returns (out fp32 [B,Hq,d], lse fp32 [B,Hq])."""
    q = _cuda(q, "q")
    k_new = _cuda(k_new, "k_new")
    v_new = _cuda(v_new, "v_new")
    if v_new is not None and v_new.dtype != k_new.dtype:
        raise TypeError("k_new and v_new must have the same dtype")
    B, Hq, d = q.shape
    T = cache.T_cap if T is None else int(T)
    sm = 1.0 / math.sqrt(d) if sm_scale is None else float(sm_scale)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = decode_workspace(cache, Hq, T)
    seq_lens = _cuda(seq_lens, "seq_lens")
    U = _cuda(U, "U") if cache.r > 0 else None
    cs = cache.struct()
    _check("headq_decode_append", lib().headq_decode_append(
        ctypes.byref(cs), _ptr(k_new), _ptr(v_new), _dtype_code(k_new), _ptr(q), _dtype_code(q),
        Hq, _ptr(seq_lens), T, _ptr(U), sm, int(corr_sign), _ptr(out), _ptr(lse), _ptr(ws),
        ws.numel(), _stream(stream)))
    return out, lse


def headq_attn_kl(cache, q, U, k_full, v_full, T=None, seq_lens=None, sm_scale=None,
                  corr_sign=1, ws=None, stream=None):
    """Returns (kl, fisher_var, a2_vdist, dout2), each fp32 [B, Hq]."""
    q = _cuda(q, "q")
    k_full = _cuda(k_full, "k_full")
    v_full = _cuda(v_full, "v_full")
    B, Hq, d = q.shape
    T = k_full.shape[2] if T is None else int(T)
    sm = 1.0 / math.sqrt(d) if sm_scale is None else float(sm_scale)
    res = [torch.empty((B, Hq), dtype=torch.float32, device=q.device) for _ in range(4)]
    if ws is None:
        ws = attn_kl_workspace(cache, Hq, T)
    seq_lens = _cuda(seq_lens, "seq_lens")
    U = _cuda(U, "U") if cache.r > 0 else None
    cs = cache.struct()
    _check("headq_attn_kl", lib().headq_attn_kl(
        ctypes.byref(cs), _ptr(q), _dtype_code(q), Hq, _ptr(seq_lens), T, _ptr(k_full),
        _ptr(v_full), _dtype_code(k_full), _ptr(U), sm, int(corr_sign),
        *[_ptr(t) for t in res], _ptr(ws), ws.numel(), _stream(stream)))
    return tuple(res)


def headq_shard_seq_lens(seq_lens, B, T, t_lo, n, out=None, device="cuda", stream=None):
    """int32 [B] local lengths clamp(T_b - t_lo, 0, n) of a token range [t_lo, t_lo+n)."""
    seq_lens = _cuda(seq_lens, "seq_lens")
    dev = seq_lens.device if seq_lens is not None else device
    out = torch.empty(B, dtype=torch.int32, device=dev) if out is None else out
    _check("headq_shard_seq_lens", lib().headq_shard_seq_lens(
        _ptr(seq_lens), int(B), int(T), int(t_lo), int(n), _ptr(out), _stream(stream)))
    return out


def headq_merge_partials(parts, S, BH, d, part_stride, out=None, lse=None, stream=None):
    """Combine S partial decodes held in one fp32 buffer of S blocks of
    part_stride floats, each [out (BH*d) | lse (BH) | padding]; returns
    (out fp32 [BH, d], lse fp32 [BH])."""
    parts = _cuda(parts, "parts")
    if parts.dtype != torch.float32 or parts.numel() < S * part_stride:
        raise ValueError("parts must be fp32 with S * part_stride elements")
    out = torch.empty((BH, d), dtype=torch.float32, device=parts.device) if out is None else out
    lse = torch.empty(BH, dtype=torch.float32, device=parts.device) if lse is None else lse
    _check("headq_merge_partials", lib().headq_merge_partials(
        _ptr(parts), ctypes.c_void_p(parts.data_ptr() + 4 * BH * d), int(S), int(BH), int(d),
        int(part_stride), _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


def a2_workspace(cache, n_obs, Hq, T):
    cs = cache.struct()
    n = lib().headq_a2_workspace_bytes(ctypes.byref(cs), n_obs, Hq, T)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=cache.k_codes.device)


def headq_a2_scores(cache, q_obs, k_full, v_full, T=None, seq_lens=None, sm_scale=None,
                    ws=None, out=None, stream=None):
    """A^2 policy scores a_j fp32 [B, Hkv, T] from observation queries
    q_obs [B, n_obs, Hq, d] and the exact keys/values [B, Hkv, T, d]."""
    q_obs = _cuda(q_obs, "q_obs")
    k_full = _cuda(k_full, "k_full")
    v_full = _cuda(v_full, "v_full")
    seq_lens = _cuda(seq_lens, "seq_lens")
    B, n_obs, Hq, d = q_obs.shape
    T = k_full.shape[2] if T is None else int(T)
    sm = 1.0 / math.sqrt(d) if sm_scale is None else float(sm_scale)
    ws = a2_workspace(cache, n_obs, Hq, T) if ws is None else ws
    out = torch.empty((cache.B, cache.Hkv, T), dtype=torch.float32,
                      device=q_obs.device) if out is None else out
    cs = cache.struct()
    _check("headq_a2_scores", lib().headq_a2_scores(
        ctypes.byref(cs), _ptr(q_obs), _dtype_code(q_obs), n_obs, Hq, _ptr(seq_lens), T,
        _ptr(k_full), _ptr(v_full), _dtype_code(k_full), ctypes.c_float(sm), _ptr(out),
        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def headq_a2_select(scores, K, v_full, seq_lens=None, keep_idx=None, keep_v=None, stream=None):
    """Top-K kept positions (int32 [B, Hkv, K], ascending, -1 padded) and their
    exact values [B, Hkv, K, d] (v_full's dtype)."""
    scores = _cuda(scores, "scores")
    v_full = _cuda(v_full, "v_full")
    seq_lens = _cuda(seq_lens, "seq_lens")
    B, Hkv, T = scores.shape
    d = v_full.shape[-1]
    keep_idx = torch.empty((B, Hkv, K), dtype=torch.int32,
                           device=scores.device) if keep_idx is None else keep_idx
    keep_v = torch.empty((B, Hkv, K, d), dtype=v_full.dtype,
                         device=scores.device) if keep_v is None else keep_v
    _check("headq_a2_select", lib().headq_a2_select(
        _ptr(scores), B, Hkv, _ptr(seq_lens), T, int(K), _ptr(v_full), _dtype_code(v_full), d,
        _ptr(keep_idx), _ptr(keep_v), _stream(stream)))
    return keep_idx, keep_v


def headq_a2_value_fixup(cache, q, U, keep_idx, keep_v, out, lse, T=None, seq_lens=None,
                         sm_scale=None, corr_sign=1, stream=None):
    """out += the kept tokens' exact-minus-cached value readout (after a decode
    that wrote out and lse with the same arguments)."""
    q = _cuda(q, "q")
    keep_idx = _cuda(keep_idx, "keep_idx")
    keep_v = _cuda(keep_v, "keep_v")
    seq_lens = _cuda(seq_lens, "seq_lens")
    B, Hq, d = q.shape
    T = cache.T_cap if T is None else int(T)
    sm = 1.0 / math.sqrt(d) if sm_scale is None else float(sm_scale)
    U = _cuda(U, "U") if cache.r > 0 else None
    cs = cache.struct()
    _check("headq_a2_value_fixup", lib().headq_a2_value_fixup(
        ctypes.byref(cs), _ptr(q), _dtype_code(q), Hq, _ptr(seq_lens), T, _ptr(U),
        ctypes.c_float(sm), int(corr_sign), _ptr(keep_idx), _ptr(keep_v), _dtype_code(keep_v),
        keep_idx.shape[-1], _ptr(out), _ptr(lse), _stream(stream)))
    return out


# The packed-batch calls are made once per layer and step, often on work of a few
# microseconds: their argument handling below keeps to plain integers, and enters a device
# guard only when the cache is on another device than the current one.

def _same_device(cache, tensors):
    """The index of the cache's device, on which every tensor of a call must be."""
    dev = cache.k_codes.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("a tensor is on %s, the cache on %s" % (t.device, cache.k_codes.device))
    return dev


def _call(name, dev, stream, *args):
    """Entry point `name` on device `dev` and its current stream (or `stream`)."""
    fn = getattr(_lib or lib(), name)
    if stream is not None and stream.device_index != dev:
        raise ValueError("the stream is on cuda:%d, the cache on cuda:%d" % (stream.device_index, dev))
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != 0:
        raise HeadQError(name, st)


def _zeros(shape, dtype, device, stream):
    """Zeros made on the stream that the call runs on."""
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        return torch.zeros(shape, dtype=dtype, device=device)


def _rows(t, name, heads, d, written=False):
    """``headq_rows`` of a packed tensor [rows, heads, d]: any row and head strides that are
    multiples of 16 bytes, channels contiguous; elements of a written one do not overlap."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError("%s must be [rows, %d, %d], got %s" % (name, heads, d, list(shape)))
    rows, code = shape[0], _dtype_code(t)
    rs, hs, cs = t.stride() if rows else (0, 0, 1)  # no rows: whatever the strides are
    per = 4 if code == HEADQ_F32 else 8
    if rows <= 1:  # the strides of a single row or head are never used
        rs = 0
    if heads == 1:
        hs = 0
    if cs != 1 or rs % per or hs % per:
        raise ValueError("%s: channels must be contiguous and the other strides multiples of 16 bytes"
                         % name)
    if written and rows and not (rs >= heads * hs >= heads * d):  # not the plain order: what lies inside what
        if rows > 1 and heads > 0:
            lo, hi = sorted(((rs, rows), (hs, heads))) if heads > 1 else ((d, 1), (rs, rows))
            if lo[0] < d or hi[0] < (lo[1] - 1) * lo[0] + d:
                raise ValueError("%s: its rows and heads overlap" % name)
        elif heads > 1 and hs < d:
            raise ValueError("%s: its rows and heads overlap" % name)
    return RowsStruct(t.data_ptr(), code, rs, hs)


def _int32(t, name, shape):
    if t is None:
        return None
    if _cuda(t, name).dtype != torch.int32 or t.shape != shape:
        raise ValueError("%s must be int32 %s" % (name, list(shape)))
    return t.data_ptr()


def _fits(T, n, rows=0):
    """The sizes fit the C structures; ctypes would wrap larger ones."""
    if not (-0x80000000 <= T <= 0x7fffffff and -0x80000000 <= n <= 0x7fffffff and rows <= 0x7fffffff):
        raise ValueError("T = %d, n = %d, %d rows: more than 32 bits" % (T, n, rows))


def _span(cache, seq_lens, cu, n, T, rows):
    """``headq_span`` of a packed batch of `rows` rows."""
    if n is None:
        if cu is not None:
            raise ValueError("n (the most rows of one sequence) is needed with cu")
        if cache.B and rows % cache.B:
            raise ValueError("%d rows are no whole number for each of %d sequences" % (rows, cache.B))
        n = rows // cache.B if cache.B else 0
    n, T = int(n), cache.T_cap if T is None else int(T)
    _fits(T, n, rows)
    return SpanStruct(_int32(seq_lens, "seq_lens", (cache.B,)), _int32(cu, "cu", (cache.B + 1,)), T, n, rows)


def _basis(cache, U):
    if cache.r == 0:
        return None
    if _cuda(U, "U") is None or U.dtype != torch.float32 or U.shape != (cache.Hkv, cache.d, cache.r):
        raise ValueError("U must be float32 [%d, %d, %d]" % (cache.Hkv, cache.d, cache.r))
    return U.data_ptr()


def headq_cache_write_ragged(cache, k, v, U, seq_lens=None, cu=None, n=None, T=None, src=None,
                             stream=None):
    """Encode a packed batch of new tokens, k and v [rows, Hkv, d] (v None: values left as
    they are), into the last cached positions of every sequence.

    Sequence b's tokens are rows cu[b] .. cu[b+1] (cu None: n rows each, n = rows / B);
    they lie at positions T_b - n_b .. T_b - 1, T_b = seq_lens[b] (None: T, or the capacity).
    n: the most rows of one sequence.  src (int32 [rows]): row r takes its token from row
    src[r] of k and v.  Strided k and v (slices of a fused projection) need no copy."""
    ks = _rows(k, "k", cache.Hkv, cache.d)
    vs = None if v is None else _rows(v, "v", cache.Hkv, cache.d)
    if v is not None and (v.dtype != k.dtype or v.shape[0] != k.shape[0]):
        raise ValueError("k and v must have the same dtype and rows")
    rows = k.shape[0] if src is None else src.shape[0]
    dev = _same_device(cache, (k, v, U, seq_lens, cu, src))
    sp = _span(cache, seq_lens, cu, n, T, rows)
    _call("headq_cache_write_ragged", dev, stream, cache.struct(), ks, vs, k.shape[0],
          _int32(src, "src", (rows,)), sp, _basis(cache, U))


def headq_cache_read(cache, U, seq_lens=None, cu=None, n=None, T=None, rows=None, corr_sign=1,
                     dtype=torch.bfloat16, k_out=None, v_out=None, ws=None, stream=None):
    """Decode cached tokens to dense (k, v), each [rows, Hkv, d]: the key the corrected logit
    reads and the cached value.  The tokens are named as in :func:`headq_cache_write_ragged`;
    any interval [a, e) of a sequence is T_b = e with n_b = e - a.  Give k_out and/or v_out
    (strided rows are fine; only what is given is computed), or neither, for new tensors of
    `dtype` with `rows` rows (B * n where there is no cu).  ws: a decode or tree workspace
    whose error word a block-table entry outside the pool sets."""
    if k_out is None and v_out is None:
        if rows is None:
            if cu is not None or n is None:
                raise ValueError("rows is needed (with cu), or n")
            rows = cache.B * n
        shape = (rows, cache.Hkv, cache.d)
        k_out, v_out = (_zeros(shape, dtype, cache.k_codes.device, stream) for _ in "kv")
    have = [t.shape[0] for t in (k_out, v_out) if t is not None]
    if len(set(have)) > 1 or (rows is not None and rows != have[0]):
        raise ValueError("k_out and v_out must have the same rows")
    ks = None if k_out is None else _rows(k_out, "k_out", cache.Hkv, cache.d, True)
    vs = None if v_out is None else _rows(v_out, "v_out", cache.Hkv, cache.d, True)
    dev = _same_device(cache, (k_out, v_out, U, seq_lens, cu, ws))
    sp = _span(cache, seq_lens, cu, n, T, have[0])
    _call("headq_cache_read", dev, stream, cache.struct(), sp, None if k_out is None else _basis(cache, U),
          int(corr_sign), ks, vs, None if ws is None else ws.data_ptr())
    return k_out, v_out


def tree_workspace(cache, Hq, n, T=None, stream=None):
    """A zeroed device workspace for headq_tree_attn with up to n new tokens per sequence and
    lengths up to T (None: the capacity)."""
    cs = cache.struct()
    n, T = int(n), cache.T_cap if T is None else int(T)
    _fits(T, n)
    with torch.cuda.device(cache.k_codes.device):
        nb = lib().headq_tree_workspace_bytes(cs, Hq, n, T)
    return _zeros(max(nb, 256), torch.uint8, cache.k_codes.device, stream)


def headq_tree_attn(cache, q, U, mask=None, seq_lens=None, cu=None, n=None, T=None, sm_scale=None,
                    corr_sign=1, out=None, lse=None, ws=None, stream=None):
    """Attention of a packed batch of new tokens q [rows, Hq, d] over the cache, which holds
    those tokens already; returns out [rows, Hq, d] of q's dtype.

    The tokens are named as in :func:`headq_cache_write_ragged`.  New token i of a sequence
    sees all tokens before its sequence's new ones, and new token j where mask[i, j] (bool or
    uint8 [n, n], one tree for all, or [B, n, n]); mask None: j <= i.  A row that sees nothing
    gives 0.  lse: fp32 [rows, Hq], written when given.  Rows of no sequence keep what `out`
    holds (zeros when it is allocated here)."""
    if q.dim() != 3:
        raise ValueError("q must be [rows, Hq, %d], got %s" % (cache.d, list(q.shape)))
    rows, Hq = q.shape[:2]
    if Hq == 0 or Hq % cache.Hkv:
        raise ValueError("Hq must be a multiple of Hkv")
    if out is None:
        out = _zeros((rows, Hq, cache.d), q.dtype, q.device, stream)
    qs, os_ = _rows(q, "q", Hq, cache.d), _rows(out, "out", Hq, cache.d, True)
    if out.shape[0] != rows or out.dtype != q.dtype:
        raise ValueError("out must have q's rows and dtype")
    if lse is not None and (_cuda(lse, "lse").dtype != torch.float32 or tuple(lse.shape) != (rows, Hq)):
        raise ValueError("lse must be float32 [%d, %d]" % (rows, Hq))
    dev = _same_device(cache, (q, out, U, mask, seq_lens, cu, lse, ws))
    sp = _span(cache, seq_lens, cu, n, T, rows)
    mp, ms = None, 0
    if mask is not None:
        if _cuda(mask, "mask").dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be bool or uint8")
        if tuple(mask.shape) == (cache.B, sp.n, sp.n):
            ms = sp.n * sp.n
        elif tuple(mask.shape) != (sp.n, sp.n):
            raise ValueError("mask must be [%d, %d] or [%d, %d, %d]" % (sp.n, sp.n, cache.B, sp.n, sp.n))
        mp = mask.data_ptr()
    if ws is None:
        ws = tree_workspace(cache, Hq, sp.n, sp.T, stream)
    sm = 1.0 / math.sqrt(cache.d) if sm_scale is None else float(sm_scale)
    _call("headq_tree_attn", dev, stream, cache.struct(), qs, Hq, mp, ms, sp, _basis(cache, U), sm,
          int(corr_sign), os_, None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def headq_workspace_status(ws, stream=None):
    """Synchronises and raises HeadQError if a kernel flagged a device-side error."""
    s = torch.cuda.current_stream(ws.device) if stream is None else stream
    with torch.cuda.device(ws.device):
        _check("headq_workspace_status",
               lib().headq_workspace_status(_ptr(ws), ctypes.c_void_p(s.cuda_stream)))
