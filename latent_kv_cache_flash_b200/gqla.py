"""ctypes binding of libgqla.so (declared in include/gqla.h).

Argument marshalling only: every step of the decode path runs in the
library's CUDA kernels.  torch tensors supply device pointers, the current
CUDA stream and, when the caller passes none, the workspace buffer.  The
functions keep the C names; a non-OK status raises :class:`GqlaError`.
There is no fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import math
import operator
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgqla.so")

GQLA_OK, GQLA_ERR_INVALID_ARG, GQLA_ERR_UNSUPPORTED, GQLA_ERR_ALIGNMENT, GQLA_ERR_WORKSPACE, GQLA_ERR_CUDA = range(6)
GQLA_F32, GQLA_BF16 = 0, 1
GQLA_PATH_ABSORB, GQLA_PATH_GQA = 0, 1
GQLA_K_PER_GROUP, GQLA_K_SHARED_ROPE = 0, 1
DEV_SHORT_SEQ, DEV_OVERFLOW, DEV_BAD_PAGE, DEV_TIMEOUT, DEV_BAD_TREE, DEV_BAD_PROBS = 1, 2, 4, 8, 16, 32
GQLA_MAX_TREE = 64


class GqlaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class GqlaDims(ctypes.Structure):
    _fields_ = [("n_h", ctypes.c_int32), ("G", ctypes.c_int32), ("d_nope", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("d_v", ctypes.c_int32), ("r", ctypes.c_int32),
                ("s_q", ctypes.c_int32), ("scale", ctypes.c_float), ("dtype", ctypes.c_int),
                ("k_layout", ctypes.c_int32)]


class GqlaKvLayout(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seq_lens", ctypes.c_void_p), ("max_seq_len", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("capacity", ctypes.c_int32), ("block_table", ctypes.c_void_p),
                ("max_blocks_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


class GqlaHw(ctypes.Structure):
    _fields_ = [("sms", ctypes.c_int32), ("hbm_gbs", ctypes.c_double), ("tc_tflops", ctypes.c_double)]


class GqlaPathEstimate(ctypes.Structure):
    _fields_ = [("absorb_us", ctypes.c_double), ("gqa_us", ctypes.c_double), ("path", ctypes.c_int)]


class GqlaTree(ctypes.Structure):
    _fields_ = [("masks", ctypes.c_void_p), ("sizes", ctypes.c_void_p)]


class GqlaPool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


_lib = None


def lib():
    """Loads libgqla.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError("libgqla.so not built: run python -m latent_kv_cache_flash_b200.build")
        L = ctypes.CDLL(_LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        pd, pl = ctypes.POINTER(GqlaDims), ctypes.POINTER(GqlaKvLayout)
        L.gqla_expand_cache.argtypes = [pd, pl, P, P, P, P, P, I32, P, P]
        L.gqla_decode_absorb.argtypes = [pd, pl, P, P, P, P, P, P, I32, P, SZ, P, P]
        L.gqla_decode_gqa.argtypes = [pd, pl, P, P, P, P, P, I32, P, SZ, P, P]
        L.gqla_decode_gqa_noalloc.argtypes = [pd, pl, P, P, P, P, P, I32, P, P]
        L.gqla_splitkv_combine.argtypes = [I32, I32, I32, P, P, P, ctypes.c_int, P, P]
        L.gqla_append_tokens.argtypes = [pd, pl, P, P, P, P, P, P, P, P]
        pt = ctypes.POINTER(GqlaTree)
        L.gqla_tree_masks.argtypes = [I32, I32, P, P, P, P, P]
        L.gqla_append_tree.argtypes = [pd, pl, P, P, P, P, P, P, P, P, P]
        L.gqla_decode_tree_gqa.argtypes = [pd, pl, pt, P, P, P, P, P, I32, P, SZ, P, P]
        L.gqla_decode_tree_absorb.argtypes = [pd, pl, pt, P, P, P, P, P, P, I32, P, SZ, P, P]
        L.gqla_tree_workspace_bytes.argtypes = [pd, pl, I32, ctypes.c_int]
        L.gqla_tree_workspace_bytes.restype = SZ
        L.gqla_tree_num_splits.argtypes = [pd, pl, I32, ctypes.c_int]
        L.gqla_tree_num_splits.restype = I32
        L.gqla_verify_tree.argtypes = [I32, I32, I32, P, P, P, P, ctypes.c_int64, P, ctypes.c_int64, ctypes.c_int, P, P,
                                       P, P, P, P, P]
        L.gqla_commit_tree.argtypes = [pl, I32, P, P, P, P, I32, P, P, P]
        L.gqla_select_path.argtypes = [pd, pl, ctypes.c_int64, ctypes.POINTER(GqlaHw),
                                       ctypes.POINTER(GqlaPathEstimate)]
        L.gqla_workspace_bytes.argtypes = [pd, pl, I32, ctypes.c_int]
        L.gqla_workspace_bytes.restype = SZ
        L.gqla_num_splits.argtypes = [pd, pl, I32, ctypes.c_int]
        L.gqla_num_splits.restype = I32
        L.gqla_cache_bytes_per_token.argtypes = [pd, ctypes.c_int]
        L.gqla_cache_bytes_per_token.restype = SZ
        L.gqla_status_string.argtypes = [ctypes.c_int]
        L.gqla_status_string.restype = ctypes.c_char_p
        L.gqla_version.restype = ctypes.c_char_p
        L.gqla_launch_counter.restype = ctypes.c_uint64
        for name in ("gqla_expand_cache", "gqla_decode_absorb", "gqla_decode_gqa", "gqla_decode_gqa_noalloc",
                     "gqla_splitkv_combine", "gqla_append_tokens", "gqla_select_path", "gqla_tree_masks",
                     "gqla_append_tree", "gqla_decode_tree_gqa", "gqla_decode_tree_absorb", "gqla_verify_tree",
                     "gqla_commit_tree"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    if stream is not None:
        return ctypes.c_void_p(stream)
    if device is not None and device.type == "cuda":
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    return None


def _allocating_on(stream, device):
    """Context in which a call's own workspace is allocated: torch hands a
    freed block to later allocations of the same stream, so it has to belong
    to the stream whose kernels still use it when the call returns."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    handle = getattr(stream, "value", stream) or 0
    if handle == torch.cuda.current_stream(device).cuda_stream:
        return contextlib.nullcontext()
    # torch takes an external handle of 0 for none
    return torch.cuda.stream(torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device))


def _check(status: int, what: str):
    if status != GQLA_OK:
        raise GqlaError(status, "%s: %s" % (what, gqla_status_string(status)))


def make_dims(d) -> GqlaDims:
    """Builds the C struct from any object with n_h, G, d_nope, d_rope, d_v, r,
    s_q, softmax_scale (or scale), dtype ("f32"/"bf16") and optionally
    k_shared_rope (the expanded K pool stores the RoPE key once per token)."""
    scale = getattr(d, "softmax_scale", None)
    if scale is None:
        scale = d.scale
    dt = GQLA_F32 if d.dtype in ("f32", torch.float32) else GQLA_BF16
    kl = GQLA_K_SHARED_ROPE if getattr(d, "k_shared_rope", False) else GQLA_K_PER_GROUP
    return GqlaDims(d.n_h, d.G, d.d_nope, d.d_rope, d.d_v, d.r, d.s_q, float(scale), dt, kl)


def make_layout(seq_lens: torch.Tensor, max_seq_len: int, page_size: int = 0, capacity: int = 0,
                block_table: Optional[torch.Tensor] = None, num_pages: int = 0) -> GqlaKvLayout:
    """seq_lens and block_table are int32 device tensors (kept alive by the caller)."""
    mbps = 0 if block_table is None else int(block_table.shape[1])
    lay = GqlaKvLayout(int(seq_lens.shape[0]), _ptr(seq_lens), int(max_seq_len), int(page_size),
                       int(capacity), _ptr(block_table), mbps, int(num_pages))
    lay._device = seq_lens.get_device()
    return lay


def gqla_status_string(status: int) -> str:
    return lib().gqla_status_string(status).decode()


def gqla_version() -> str:
    return lib().gqla_version().decode()


def gqla_launch_counter() -> int:
    return int(lib().gqla_launch_counter())


def gqla_cache_bytes_per_token(dims: GqlaDims, path: int) -> int:
    return int(lib().gqla_cache_bytes_per_token(ctypes.byref(dims), path))


def gqla_workspace_bytes(dims: GqlaDims, layout: GqlaKvLayout, num_splits: int, path: int) -> int:
    return int(lib().gqla_workspace_bytes(ctypes.byref(dims), ctypes.byref(layout), num_splits, path))


def gqla_num_splits(dims: GqlaDims, layout: GqlaKvLayout, num_splits: int, path: int) -> int:
    return int(lib().gqla_num_splits(ctypes.byref(dims), ctypes.byref(layout), num_splits, path))


def gqla_select_path(dims: GqlaDims, layout: GqlaKvLayout, total_tokens: int, hw: Optional[GqlaHw] = None):
    """(path, absorb_us, gqa_us): the library's prediction of both decode calls."""
    est = GqlaPathEstimate()
    s = lib().gqla_select_path(ctypes.byref(dims), ctypes.byref(layout), int(total_tokens),
                               ctypes.byref(hw) if hw is not None else None, ctypes.byref(est))
    _check(s, "gqla_select_path")
    return int(est.path), float(est.absorb_us), float(est.gqa_us)


def workspace_for(dims: GqlaDims, layout: GqlaKvLayout, num_splits: int, path: int, device) -> torch.Tensor:
    n = gqla_workspace_bytes(dims, layout, num_splits, path)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def gqla_expand_cache(dims, layout, latent, W_uk, W_uv, k_pool, v_pool, tail_tokens=0, dev_status=None,
                      stream=None):
    """Expand every cached token (or, with tail_tokens > 0, only each
    sequence's last tail_tokens) into the per-group pools: K rows
    [c_KV W_uk^g ; k_rope], V rows c_KV W_uv^g.  Pools share the latent pool's
    geometry (contiguous or paged through the same block table)."""
    s = lib().gqla_expand_cache(ctypes.byref(dims), ctypes.byref(layout), _ptr(latent), _ptr(W_uk), _ptr(W_uv),
                                _ptr(k_pool), _ptr(v_pool), int(tail_tokens), _ptr(dev_status),
                                _stream(stream, latent.device))
    _check(s, "gqla_expand_cache")


def gqla_append_tokens(dims, layout, new_rows, latent, W_uk=None, W_uv=None, k_pool=None, v_pool=None,
                       dev_status=None, stream=None):
    """Write each sequence's s_q new token rows new_rows [B, s_q, r + d_rope]
    at positions seq_len - s_q .. seq_len - 1: into the latent pool (when
    latent is given) and, expanded, into the per-group pools (when k_pool and
    v_pool are given; W_uk and W_uv are then required).  latent=None expands
    only, reading the rows from new_rows."""
    s = lib().gqla_append_tokens(ctypes.byref(dims), ctypes.byref(layout), _ptr(new_rows), _ptr(latent), _ptr(W_uk),
                                 _ptr(W_uv), _ptr(k_pool), _ptr(v_pool), _ptr(dev_status),
                                 _stream(stream, new_rows.device))
    _check(s, "gqla_append_tokens")


def gqla_decode_absorb(dims, layout, q, latent, W_uk, W_uv, out, lse=None, num_splits=0, workspace=None,
                       dev_status=None, stream=None):
    """Absorb-path decode over the latent pool: q_nope is absorbed into the
    latent space per group, scores run against [c_KV ; k_rope], the latent
    output is up-projected by W_uv.  out [B, s_q, n_h, d_v]; lse [B, s_q, n_h]
    fp32 (natural log) when given.  num_splits 0 takes the library's plan; a
    workspace of gqla_workspace_bytes is allocated when none is passed."""
    if workspace is None:
        with _allocating_on(stream, q.device):
            workspace = workspace_for(dims, layout, num_splits, GQLA_PATH_ABSORB, q.device)
    s = lib().gqla_decode_absorb(ctypes.byref(dims), ctypes.byref(layout), _ptr(q), _ptr(latent), _ptr(W_uk),
                                 _ptr(W_uv), _ptr(out), _ptr(lse), int(num_splits), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                 _stream(stream, q.device))
    _check(s, "gqla_decode_absorb")


def gqla_decode_gqa(dims, layout, q, k_pool, v_pool, out, lse=None, num_splits=0, workspace=None,
                    dev_status=None, stream=None):
    """GQA-path decode over the expanded per-group pools: each group's m heads
    attend to that group's K/V rows.  Same output, lse, split and workspace
    conventions as gqla_decode_absorb."""
    if workspace is None:
        with _allocating_on(stream, q.device):
            workspace = workspace_for(dims, layout, num_splits, GQLA_PATH_GQA, q.device)
    s = lib().gqla_decode_gqa(ctypes.byref(dims), ctypes.byref(layout), _ptr(q), _ptr(k_pool), _ptr(v_pool),
                              _ptr(out), _ptr(lse), int(num_splits), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(dev_status),
                              _stream(stream, q.device))
    _check(s, "gqla_decode_gqa")


def gqla_decode_gqa_noalloc(dims, layout, q, k_pool, v_pool, out, lse=None, num_splits=0, dev_status=None,
                            stream=None):
    """gqla_decode_gqa with its split scratch in the library's own fixed device
    array: no workspace, no allocation (see include/gqla.h for the limit)."""
    s = lib().gqla_decode_gqa_noalloc(ctypes.byref(dims), ctypes.byref(layout), _ptr(q), _ptr(k_pool),
                                      _ptr(v_pool), _ptr(out), _ptr(lse), int(num_splits), _ptr(dev_status),
                                      _stream(stream, q.device))
    _check(s, "gqla_decode_gqa_noalloc")


def gqla_splitkv_combine(o_part, lse_part, out, lse_out=None, stream=None):
    S, rows, D = (int(x) for x in o_part.shape)
    dt = GQLA_F32 if out.dtype == torch.float32 else GQLA_BF16
    s = lib().gqla_splitkv_combine(S, rows, D, _ptr(o_part), _ptr(lse_part), _ptr(out), dt, _ptr(lse_out),
                                   _stream(stream, o_part.device))
    _check(s, "gqla_splitkv_combine")


# ---- speculative decoding with a tree of drafted tokens ------------------


def _require(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def _plain(t: Optional[torch.Tensor], dtype, shape, dev: int, name: str):
    """A contiguous tensor of this type and shape on this device, or None."""
    if t is not None and not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev):
        raise ValueError("%s: contiguous %s %s on the call's device expected" % (name, dtype, list(shape)))


def _dense(dev: int, expected):
    """Contiguous tensors on this device; expected: (tensor, dtype, elements,
    name), a negative number for "at least"; a tensor may be None."""
    for t, dtype, n, name in expected:
        if t is None:
            continue
        size = t.numel()
        if not ((size == n or 0 <= -n <= size) and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev):
            raise ValueError("%s: %s%d contiguous elements of %s on the call's device expected" %
                             (name, "at least " if n < 0 else "", abs(n), dtype))


def _status(t: Optional[torch.Tensor], dev: int):
    if t is not None:
        _dense(dev, ((t, torch.int32, -1, "dev_status"),))


def _on_layouts_device(layout, dev: int):
    if getattr(layout, "_device", dev) != dev:
        raise ValueError("layout: lengths on the call's device expected")


def _rows(layout) -> int:
    """Token rows of a pool."""
    per = layout.page_size
    return layout.num_pages * per if per else layout.batch * layout.capacity


def _element(dims):
    return torch.float32 if dims.dtype == GQLA_F32 else torch.bfloat16


def _expanded(dims, dt, rows: int, k_pool, v_pool):
    G, r = dims.G, dims.d_rope
    return ((k_pool, dt, -rows * (G * dims.d_nope + (r if dims.k_layout == GQLA_K_SHARED_ROPE else G * r)), "k_pool"),
            (v_pool, dt, -rows * G * dims.d_v, "v_pool"))


def _weights(dims, dt, W_uk, W_uv):
    per = dims.G * dims.r
    return (W_uk, dt, per * dims.d_nope, "W_uk"), (W_uv, dt, per * dims.d_v, "W_uv")


def _attention(dims, dt, layout, tree, q, out, lse, workspace, dev_status, model):
    """Checks the tensors of a tree attention call."""
    dev = q.get_device()
    _on_layouts_device(layout, dev)
    B, T = layout.batch, dims.s_q
    slots = getattr(tree, "_slots", None)
    if slots is not None and slots != (B, T, dev):
        raise ValueError("tree: masks [%d, %d] on the call's device expected" % (B, T))
    rows = B * T * dims.n_h
    _dense(dev, ((q, dt, rows * (dims.d_nope + dims.d_rope), "q"), (out, dt, rows * dims.d_v, "out"),
                 (lse, torch.float32, rows, "lse"), (dev_status, torch.int32, -1, "dev_status")) + model)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace: contiguous on the call's device expected")


# The current stream's handle without a Stream object around it, which costs a
# tenth of a small call; where torch has none, through the object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(what: str, fn, tensor: torch.Tensor, stream, *args):
    """fn(*args, stream) on the tensor's device, whichever one is current."""
    if tensor.is_cuda:
        dev = tensor.get_device()
        if dev == torch.cuda.current_device():
            s = fn(*args, _raw_stream(dev) if stream is None else stream)
        else:
            with torch.cuda.device(dev):
                s = fn(*args, _raw_stream(dev) if stream is None else stream)
    else:
        s = fn(*args, stream)
    if s != GQLA_OK:
        _check(s, what)


def make_tree(masks: torch.Tensor, sizes: Optional[torch.Tensor] = None) -> GqlaTree:
    """masks [B, s_q] (64-bit words) and sizes [B] int32 are device tensors
    kept alive by the caller; sizes None: every sequence drafted s_q tokens."""
    _require(masks.dtype in (torch.int64, torch.uint64) and masks.dim() == 2 and masks.is_contiguous(),
             "masks: contiguous 64-bit words [batch, tokens] expected")
    dev = masks.get_device()
    _plain(sizes, torch.int32, masks.shape[:1], dev, "sizes")
    tree = GqlaTree(_ptr(masks), _ptr(sizes))
    tree._slots = (*masks.shape, dev)
    return tree


def gqla_tree_masks(parents, masks, sizes=None, dev_status=None, stream=None):
    """masks[b, i] = bits of drafted token i and its ancestors, from
    parents [B, n_tokens] int32 (parents[b, i] < i, -1 for a root)."""
    _require(parents.dim() == 2, "parents: [batch, tokens] expected")
    dev = parents.get_device()
    _plain(parents, torch.int32, parents.shape, dev, "parents")
    _plain(sizes, torch.int32, parents.shape[:1], dev, "sizes")
    _require(masks.dtype in (torch.int64, torch.uint64) and masks.shape == parents.shape and masks.is_contiguous() and
             masks.get_device() == dev, "masks: contiguous 64-bit words of the parents' shape expected")
    _status(dev_status, dev)
    B, T = parents.shape
    _call("gqla_tree_masks", lib().gqla_tree_masks, parents, stream, B, T, _ptr(parents), _ptr(sizes), _ptr(masks),
          _ptr(dev_status))


def gqla_append_tree(dims, layout, new_rows, latent, W_uk=None, W_uv=None, k_pool=None, v_pool=None, sizes=None,
                     dev_status=None, stream=None):
    """gqla_append_tokens for the drafted tokens: rows new_rows[b, i],
    i < sizes[b], go to positions seq_len - sizes[b] + i."""
    dev = new_rows.get_device()
    _on_layouts_device(layout, dev)
    _plain(sizes, torch.int32, (layout.batch,), dev, "sizes")
    dt, rows, width = _element(dims), _rows(layout), dims.r + dims.d_rope
    _dense(dev, ((new_rows, dt, layout.batch * dims.s_q * width, "new_rows"), (latent, dt, -rows * width, "latent")))
    if k_pool is not None or v_pool is not None:
        _dense(dev, _expanded(dims, dt, rows, k_pool, v_pool) + _weights(dims, dt, W_uk, W_uv))
    _status(dev_status, dev)
    _call("gqla_append_tree", lib().gqla_append_tree, new_rows, stream, ctypes.byref(dims), ctypes.byref(layout),
          _ptr(sizes), _ptr(new_rows), _ptr(latent), _ptr(W_uk), _ptr(W_uv), _ptr(k_pool), _ptr(v_pool),
          _ptr(dev_status))


def gqla_tree_workspace_bytes(dims: GqlaDims, layout: GqlaKvLayout, num_splits: int, path: int) -> int:
    return int(lib().gqla_tree_workspace_bytes(ctypes.byref(dims), ctypes.byref(layout), num_splits, path))


def gqla_tree_num_splits(dims: GqlaDims, layout: GqlaKvLayout, num_splits: int, path: int) -> int:
    return int(lib().gqla_tree_num_splits(ctypes.byref(dims), ctypes.byref(layout), num_splits, path))


def tree_workspace_for(dims: GqlaDims, layout: GqlaKvLayout, num_splits: int, path: int, device) -> torch.Tensor:
    n = gqla_tree_workspace_bytes(dims, layout, num_splits, path)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def gqla_decode_tree_gqa(dims, layout, tree, q, k_pool, v_pool, out, lse=None, num_splits=0, workspace=None,
                         dev_status=None, stream=None):
    """Attention of a tree of drafted tokens over the expanded per-group
    pools: token i of sequence b sees every token before the tree and the
    drafted tokens of tree.masks[b, i].  out [B, s_q, n_h, d_v], lse
    [B, s_q, n_h]; rows of slots past a sequence's tree are 0 and -inf.
    num_splits is used by the forms without tensor cores only."""
    dt = _element(dims)
    _attention(dims, dt, layout, tree, q, out, lse, workspace, dev_status,
               _expanded(dims, dt, _rows(layout), k_pool, v_pool))
    if workspace is None:
        with _allocating_on(stream, q.device):
            workspace = tree_workspace_for(dims, layout, num_splits, GQLA_PATH_GQA, q.device)
    _call("gqla_decode_tree_gqa", lib().gqla_decode_tree_gqa, q, stream, ctypes.byref(dims), ctypes.byref(layout),
          ctypes.byref(tree), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(out), _ptr(lse), int(num_splits),
          _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status))


def gqla_decode_tree_absorb(dims, layout, tree, q, latent, W_uk, W_uv, out, lse=None, num_splits=0, workspace=None,
                            dev_status=None, stream=None):
    """Attention of a tree of drafted tokens over the latent pool (the
    absorbed form); otherwise as gqla_decode_tree_gqa."""
    dt = _element(dims)
    _attention(dims, dt, layout, tree, q, out, lse, workspace, dev_status,
               ((latent, dt, -_rows(layout) * (dims.r + dims.d_rope), "latent"),) + _weights(dims, dt, W_uk, W_uv))
    if workspace is None:
        with _allocating_on(stream, q.device):
            workspace = tree_workspace_for(dims, layout, num_splits, GQLA_PATH_ABSORB, q.device)
    _call("gqla_decode_tree_absorb", lib().gqla_decode_tree_absorb, q, stream, ctypes.byref(dims),
          ctypes.byref(layout), ctypes.byref(tree), _ptr(q), _ptr(latent), _ptr(W_uk), _ptr(W_uv), _ptr(out),
          _ptr(lse), int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(),
          _ptr(dev_status))


_shape = operator.attrgetter("shape")


def _pitch(t: torch.Tensor, B: int, T: int, V: int, name: str) -> int:
    """Elements between the rows of probabilities [B, T, V], whose rows are
    evenly spaced and contiguous inside."""
    sb, st, sv = t.stride()
    pitch = st if T > 1 else sb if B > 1 else V
    if pitch < V or (V > 1 and sv != 1) or (B > 1 and T > 1 and sb != T * pitch):
        raise ValueError("%s: contiguous rows at one pitch expected" % name)
    return pitch


def gqla_verify_tree(parents, tokens, target, draft, u_accept, u_sample, accepted, n_accepted, next_token, sizes=None,
                     dev_status=None, stream=None):
    """Rejection sampling along the drafted trees: parents and tokens [B, T]
    int32; target and draft [B, T, V] probabilities after each token, both
    fp32 or both bf16 (draft None: tokens chosen for certain); u_accept
    [B, T] and u_sample [B] fp32 in [0, 1).  Written, all int32: accepted
    [B, T] (path of token indices from the root, -1 behind it), n_accepted
    [B], next_token [B]."""
    _require(target.dim() == 3, "target: [batch, tokens, vocab] expected")
    shape = target.shape
    B, T, V = shape
    dt, i32 = target.dtype, torch.int32
    _require((dt is torch.float32 or dt is torch.bfloat16) and
             (draft is None or (draft.dtype is dt and draft.shape == shape)),
             "target and draft: both fp32 or both bf16 [batch, tokens, vocab] expected")
    slots, rows = shape[:2], shape[:1]
    dev = target.get_device()
    _require(draft is None or draft.get_device() == dev, "draft: the target's device expected")
    _plain(parents, i32, slots, dev, "parents")
    _plain(tokens, i32, slots, dev, "tokens")
    _plain(accepted, i32, slots, dev, "accepted")
    _plain(n_accepted, i32, rows, dev, "n_accepted")
    _plain(next_token, i32, rows, dev, "next_token")
    _plain(sizes, i32, rows, dev, "sizes")
    _plain(u_accept, torch.float32, slots, dev, "u_accept")
    _plain(u_sample, torch.float32, rows, dev, "u_sample")
    _status(dev_status, dev)
    _call("gqla_verify_tree", lib().gqla_verify_tree, target, stream, B, T, V, _ptr(parents), _ptr(sizes), _ptr(tokens),
          _ptr(target), _pitch(target, B, T, V, "target"), _ptr(draft),
          0 if draft is None else _pitch(draft, B, T, V, "draft"),
          GQLA_F32 if dt is torch.float32 else GQLA_BF16, _ptr(u_accept), _ptr(u_sample),
          _ptr(accepted), _ptr(n_accepted), _ptr(next_token), _ptr(dev_status))


def gqla_commit_tree(layout, accepted, n_accepted, pools, seq_lens_out=None, sizes=None, dev_status=None,
                     stream=None):
    """Move the accepted path's rows to the positions behind the context, in
    every pool of `pools` (contiguous tensors [sequences or pages, rows,
    ...]); seq_lens_out [B] gets the new lengths."""
    pools = list(pools)
    _require(len(pools) > 0, "pools: at least one expected")
    _require(accepted.dim() == 2, "accepted: [batch, tokens] expected")
    B, T = accepted.shape
    _require(B == layout.batch, "accepted: the layout's batch expected")
    i32, rows = torch.int32, accepted.shape[:1]
    dev = accepted.get_device()
    _on_layouts_device(layout, dev)
    _plain(accepted, i32, (B, T), dev, "accepted")
    _plain(n_accepted, i32, rows, dev, "n_accepted")
    _plain(seq_lens_out, i32, rows, dev, "seq_lens_out")
    _plain(sizes, i32, rows, dev, "sizes")
    _status(dev_status, dev)
    lead = (B, layout.capacity) if layout.page_size == 0 else (layout.num_pages, layout.page_size)
    # the pools of a model's layers are alike, and there are many
    shapes = list(map(_shape, pools))
    sizes_of = list(map(torch.Tensor.element_size, pools))
    n = len(pools)
    alike = shapes.count(shapes[0]) == n and sizes_of.count(sizes_of[0]) == n
    _require(all(len(shape) >= 3 and shape[:2] == lead for shape in (shapes[:1] if alike else shapes)),
             "pools: [%d, %d, ...] of the layout expected" % lead)
    _require(all(map(torch.Tensor.is_contiguous, pools)), "pools: contiguous tensors expected")
    _require(list(map(torch.Tensor.get_device, pools)).count(dev) == n, "pools: the path's device expected")
    flat = [0] * (2 * n)
    flat[0::2] = map(torch.Tensor.data_ptr, pools)
    flat[1::2] = ([math.prod(shapes[0][2:]) * sizes_of[0]] * n if alike else
                  [math.prod(shape[2:]) * size for shape, size in zip(shapes, sizes_of)])
    arr = array.array("q", flat)      # pairs of address and row bytes: gqla_pool
    _call("gqla_commit_tree", lib().gqla_commit_tree, accepted, stream, ctypes.byref(layout), T, _ptr(sizes),
          _ptr(accepted), _ptr(n_accepted), arr.buffer_info()[0], n, _ptr(seq_lens_out), _ptr(dev_status))
