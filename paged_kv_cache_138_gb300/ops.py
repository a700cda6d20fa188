"""Python face of the libpagedkv kernels: torch tensors in, C-ABI call out.

Every function here only checks shapes and dtypes and marshals pointers; all
computation runs in the CUDA kernels of libpagedkv.so.  Device tensors must be
contiguous and live on the current CUDA device; work is enqueued on the current
torch stream unless ``stream`` (a torch.cuda.Stream or raw handle) is given.
"""
import ctypes
import functools

import torch

from ._lib import PKV_CODE_E4M3, PKV_CODE_INT8, check, lib

HEAD_DIM = 128
BLOCK_SIZE = 16


# Marshalling costs more than a small launch runs, so handles and pointers go to
# ctypes as plain integers, and the current stream is asked for without building a
# torch.cuda.Stream (2.8 us of a 14 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_handle(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_get_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t):
    return t.data_ptr() if t is not None else None


_Tensor = torch.Tensor


def _dev(t, name, dtype, ndim=None):
    if isinstance(t, _Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() and \
            (ndim is None or t.dim() == ndim):
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got %s" % (name, ndim, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


class PreparedLaunch:
    """One C-ABI launch whose arguments were checked and marshalled once.

    Calling it enqueues the same launch again: same tensors (their current
    contents), same stream.  It keeps those tensors alive.  The per-call cost
    is the C call alone, for loops that relaunch on fixed buffers (the
    ``prepare=True`` form of the launch functions below)."""

    __slots__ = ("_fn", "_args", "_what", "_keep")

    def __init__(self, fn, args, what, keep):
        self._fn, self._args, self._what, self._keep = fn, args, what, keep

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != 0:
            check(rc, self._what)


def _run(fn, args, what, prepare, keep, result):
    """Launch, or with prepare a PreparedLaunch that holds the tensors keep."""
    if prepare:
        return PreparedLaunch(fn, args, what, keep)
    rc = fn(*args)
    if rc:
        check(rc, what)
    return result


def _issue(fn, args, what, keep, prepare, result):
    if prepare:
        return PreparedLaunch(fn, args, what, keep)
    check(fn(*args), what)
    return result


def fill_normal(t, seed, offset, stream=None):
    """Fill fp16 tensor ``t`` (contiguous, 16-byte aligned) with standard-normal
    values: elements offset .. offset + numel - 1 of the device stream keyed by
    ``seed`` (``pkv_fill_normal_f16``).  Returns the offset after them."""
    _dev(t, "t", torch.float16)
    n = t.numel()
    check(lib().pkv_fill_normal_f16(_ptr(t), n, ctypes.c_uint64(seed & 0xFFFFFFFFFFFFFFFF),
                                    ctypes.c_uint64(offset), _stream_handle(stream)),
          "pkv_fill_normal_f16")
    return offset + n


def new_error_word(device=None):
    """A zeroed device int32 for the kernels' first-error code."""
    return torch.zeros(1, dtype=torch.int32, device=device or torch.cuda.current_device())


def read_error_word(dev_err):
    """Synchronise and return the device error code (0 = none)."""
    torch.cuda.current_stream().synchronize()
    return int(dev_err.item())


@functools.lru_cache(maxsize=256)
def workspace_bytes(num_seqs, num_q_heads, max_blocks_per_seq, block_size=BLOCK_SIZE,
                    head_dim=HEAD_DIM):
    """Bytes of split-K partials paged_attention_decode may need (an upper
    bound over the split lengths a launch of these sizes can choose)."""
    return int(lib().pkv_paged_attention_workspace_bytes(num_seqs, num_q_heads,
                                                         max_blocks_per_seq, block_size,
                                                         head_dim))


def split_tokens(num_seqs, num_kv_heads, max_blocks_per_seq, block_size=BLOCK_SIZE):
    """Split length (tokens) the attention launches use for these sizes."""
    t = lib().pkv_paged_attention_split_tokens(num_seqs, num_kv_heads, max_blocks_per_seq,
                                               block_size)
    if t < 0:
        check(t, "pkv_paged_attention_split_tokens")
    return t


def alloc_workspace(num_seqs, num_q_heads, max_blocks_per_seq, device=None,
                    block_size=BLOCK_SIZE):
    """A device buffer of workspace_bytes (None when no split is possible)."""
    n = workspace_bytes(num_seqs, num_q_heads, max_blocks_per_seq, block_size)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or torch.cuda.current_device())


def _new_workspace(nbytes, device, stream):
    """A workspace for one launch on ``stream``, from that stream's memory: it is given
    back when the call returns, for later work of the same stream."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else \
            torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                           workspace=None, dev_err=None, stream=None, prepare=False):
    """out[s,h] = softmax(scale * q[s,h] . K_s^T) V_s over context_lens[s] tokens.
    prepare=True returns a PreparedLaunch instead of launching."""
    _dev(q, "q", torch.float16, 3)
    _dev(out, "out", torch.float16, 3)
    _dev(k_cache, "k_cache", torch.float16, 4)
    _dev(v_cache, "v_cache", torch.float16, 4)
    _dev(block_tables, "block_tables", torch.int32, 2)
    _dev(context_lens, "context_lens", torch.int32, 1)
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_cache.shape
    if out.shape != q.shape or v_cache.shape != k_cache.shape or D2 != D:
        raise ValueError("shape mismatch")
    if block_tables.shape[0] != S or context_lens.shape[0] != S:
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    max_blocks = block_tables.shape[1]
    need = workspace_bytes(S, Hq, max_blocks, bs, D)
    if need and workspace is None:
        workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
            _ptr(context_lens), S, Hq, Hkv, D, bs, nb, max_blocks, float(scale), _ptr(workspace),
            ws_bytes, _ptr(dev_err), _stream_handle(stream))
    keep = (out, q, k_cache, v_cache, block_tables, context_lens, workspace, dev_err, stream)
    return _issue(lib().pkv_paged_attention_decode, args, "paged_attention_decode", keep, prepare,
                  out)


def paged_attention_decode_fused(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                 context_lens, scale, workspace=None, dev_err=None, stream=None,
                                 prepare=False, cow=None):
    """One launch: store k_new[s]/v_new[s] at position context_lens[s] - 1 of each
    sequence (slot from its block table) and attend over context_lens[s] tokens.
    cow=(cow_block, cow_src) (int32 [S] device tensors, see cow_targets) also
    makes each sequence's copy-on-write copy in the same launch.
    prepare=True returns a PreparedLaunch instead of launching."""
    _dev(q, "q", torch.float16, 3)
    _dev(out, "out", torch.float16, 3)
    _dev(k_new, "k_new", torch.float16, 3)
    _dev(v_new, "v_new", torch.float16, 3)
    _dev(k_cache, "k_cache", torch.float16, 4)
    _dev(v_cache, "v_cache", torch.float16, 4)
    _dev(block_tables, "block_tables", torch.int32, 2)
    _dev(context_lens, "context_lens", torch.int32, 1)
    S, Hq, D = q.shape
    nb, bs, Hkv, D2 = k_cache.shape
    if out.shape != q.shape or v_cache.shape != k_cache.shape or D2 != D:
        raise ValueError("shape mismatch")
    if k_new.shape != (S, Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new / v_new must be [num_seqs, num_kv_heads, head_dim]")
    max_blocks = block_tables.shape[1]
    need = workspace_bytes(S, Hq, max_blocks, bs, D)
    if need and workspace is None:
        workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if cow is not None:
        cb, cs = _cow_args(cow, S)
        args = (_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                _ptr(block_tables), _ptr(context_lens), _ptr(cb), _ptr(cs), S, Hq, Hkv, D, bs,
                nb, max_blocks, float(scale), _ptr(workspace), ws_bytes, _ptr(dev_err),
                _stream_handle(stream))
        keep = (out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, cb, cs,
                workspace, dev_err, stream)
        return _issue(lib().pkv_paged_attention_decode_fused_cow, args,
                      "paged_attention_decode_fused_cow", keep, prepare, out)
    args = (_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
            _ptr(block_tables), _ptr(context_lens), S, Hq, Hkv, D, bs, nb, max_blocks,
            float(scale), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream_handle(stream))
    keep = (out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, workspace,
            dev_err, stream)
    return _issue(lib().pkv_paged_attention_decode_fused, args, "paged_attention_decode_fused",
                  keep, prepare, out)


def _cow_args(cow, S):
    cb, cs = cow
    _dev(cb, "cow_block", torch.int32, 1)
    _dev(cs, "cow_src", torch.int32, 1)
    if cb.shape[0] != S or cs.shape[0] != S:
        raise ValueError("cow_block / cow_src must be int32 [num_seqs]")
    return cb, cs


def cow_targets(pairs, block_tables):
    """Host (native): copy-on-write pairs (src, dst) -> (cow_block, cow_src),
    int32 [S] numpy arrays for the fused launches' ``cow`` argument: the logical
    block of each sequence whose table holds a pair's dst, and that pair's src
    (-1 where none).  Raises PagedKVError (UNSUPPORTED) if a sequence needs
    two copies in one step."""
    import numpy as np
    pr = np.ascontiguousarray(np.asarray(pairs, dtype=np.int64).reshape(-1, 2))
    tables = np.ascontiguousarray(block_tables, dtype=np.int32)
    S = tables.shape[0]
    cb = np.empty(max(S, 1), np.int32)
    cs = np.empty(max(S, 1), np.int32)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    rc = lib().pkv_cow_targets(p(pr), pr.shape[0], p(tables), S, tables.shape[1], p(cb), p(cs))
    check(rc, "cow_targets")
    return cb[:S], cs[:S]


def reshape_and_cache(k, v, slot_mapping, k_cache, v_cache, dev_err=None, stream=None,
                      prepare=False):
    """k_cache[slot // bs, slot % bs] = k[i] (and v) for slot = slot_mapping[i] >= 0.
    prepare=True returns a PreparedLaunch instead of launching."""
    _dev(k, "k", torch.float16, 3)
    _dev(v, "v", torch.float16, 3)
    _dev(slot_mapping, "slot_mapping", torch.int64, 1)
    _dev(k_cache, "k_cache", torch.float16, 4)
    _dev(v_cache, "v_cache", torch.float16, 4)
    T, Hkv, D = k.shape
    nb, bs, Hkv2, D2 = k_cache.shape
    if v.shape != k.shape or v_cache.shape != k_cache.shape or (Hkv2, D2) != (Hkv, D):
        raise ValueError("shape mismatch")
    if slot_mapping.shape[0] != T:
        raise ValueError("slot_mapping must have one entry per token")
    args = (_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), T, Hkv, D, bs,
            nb, _ptr(dev_err), _stream_handle(stream))
    keep = (k, v, slot_mapping, k_cache, v_cache, dev_err, stream)
    return _issue(lib().pkv_reshape_and_cache, args, "reshape_and_cache", keep, prepare, None)


def slot_mapping(block_tables, positions, num_blocks, block_size=BLOCK_SIZE, out=None,
                 dev_err=None, stream=None):
    """slot[s] = table[s][p // bs] * bs + p % bs with p = positions[s] (device)."""
    _dev(block_tables, "block_tables", torch.int32, 2)
    _dev(positions, "positions", torch.int32, 1)
    S, mb = block_tables.shape
    if out is None:
        out = torch.empty(S, dtype=torch.int64, device=block_tables.device)
    _dev(out, "out", torch.int64, 1)
    rc = lib().pkv_slot_mapping(_ptr(block_tables), _ptr(positions), S, mb, block_size,
                                int(num_blocks), _ptr(out), _ptr(dev_err), _stream_handle(stream))
    check(rc, "slot_mapping")
    return out


def copy_blocks(k_caches, v_caches, block_pairs, dev_err=None, stream=None):
    """cache[dst] = cache[src] for every (src, dst) row of block_pairs, every layer."""
    if isinstance(k_caches, torch.Tensor):
        k_caches, v_caches = [k_caches], [v_caches]
    if len(k_caches) != len(v_caches) or not k_caches:
        raise ValueError("need matching, non-empty lists of K and V caches")
    _dev(block_pairs, "block_pairs", torch.int64, 2)
    ref = k_caches[0]
    for c in list(k_caches) + list(v_caches):
        _dev(c, "cache", ref.dtype)
        if c.shape != ref.shape:
            raise ValueError("all caches must share one shape")
    n = len(k_caches)
    kp = (ctypes.c_void_p * n)(*[c.data_ptr() for c in k_caches])
    vp = (ctypes.c_void_p * n)(*[c.data_ptr() for c in v_caches])
    block_bytes = ref[0].numel() * ref.element_size()
    rc = lib().pkv_copy_blocks(kp, vp, n, _ptr(block_pairs), block_pairs.shape[0], block_bytes,
                               ref.shape[0], _ptr(dev_err), _stream_handle(stream))
    check(rc, "copy_blocks")


def swap_blocks(src_pools, dst_pools, block_pairs, dev_err=None, stream=None):
    """dst_pools[i][dst] = src_pools[i][src] for every (src, dst) row of block_pairs.

    Pools are tensors of one shape per side ([num_blocks, ...]); either side may
    be pinned host memory (``tensor.is_pinned()``), which the kernel reads or
    writes over the host link.  block_pairs must be readable by the GPU (a CUDA
    tensor or pinned host memory)."""
    if isinstance(src_pools, torch.Tensor):
        src_pools, dst_pools = [src_pools], [dst_pools]
    if len(src_pools) != len(dst_pools) or not src_pools:
        raise ValueError("need matching, non-empty lists of source and destination pools")
    for side in (src_pools, dst_pools):
        for t in side:
            if not (t.is_cuda or t.is_pinned()):
                raise TypeError("pools must be CUDA tensors or pinned host tensors")
            if not t.is_contiguous() or t.shape[1:] != side[0].shape[1:]:
                raise ValueError("pools of one side must be contiguous with one shape")
    if src_pools[0][0].numel() * src_pools[0].element_size() != \
            dst_pools[0][0].numel() * dst_pools[0].element_size():
        raise ValueError("source and destination blocks differ in size")
    if block_pairs.dtype != torch.int64 or block_pairs.dim() != 2 or not \
            (block_pairs.is_cuda or block_pairs.is_pinned()):
        raise TypeError("block_pairs must be int64 [P, 2] on the GPU or pinned")
    n = len(src_pools)
    sp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in src_pools])
    dp = (ctypes.c_void_p * n)(*[t.data_ptr() for t in dst_pools])
    block_bytes = src_pools[0][0].numel() * src_pools[0].element_size()
    rc = lib().pkv_swap_blocks(sp, dp, n, _ptr(block_pairs), block_pairs.shape[0], block_bytes,
                               src_pools[0].shape[0], dst_pools[0].shape[0], _ptr(dev_err),
                               _stream_handle(stream))
    check(rc, "swap_blocks")


def shared_prefix_groups(block_tables, context_lens, block_size=BLOCK_SIZE, group_size_limit=16):
    """Host planning of grouped attention (native): consecutive sequences whose
    tables start with the same physical block form a group (at most
    group_size_limit members); a group shares the longest run of leading blocks
    every member has in common with its first member, cut to a multiple of 16
    tokens and of the block size and to the shortest member's context.

    Returns (group_first int32 [G+1], seq_group int32 [S], group_shared int32
    [G], max_shared_tokens, max_own_tokens)."""
    import numpy as np
    tables = np.ascontiguousarray(block_tables, dtype=np.int32)
    lens = np.ascontiguousarray(context_lens, dtype=np.int32)
    S = len(lens)
    first = np.empty(S + 1, np.int32)
    seq_group = np.empty(max(S, 1), np.int32)
    shared = np.empty(max(S, 1), np.int32)
    ng, ms, mo = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    rc = lib().pkv_plan_shared_prefix_groups(
        p(tables), p(lens), S, tables.shape[1] if tables.ndim == 2 else 1, int(block_size),
        int(group_size_limit), p(first), p(seq_group), p(shared), ctypes.byref(ng),
        ctypes.byref(ms), ctypes.byref(mo))
    check(rc, "plan_shared_prefix_groups")
    n = ng.value
    return first[:n + 1], seq_group[:S], shared[:n], ms.value, mo.value


def grouped_workspace_bytes(num_seqs, num_q_heads, max_blocks_per_seq, max_shared_tokens,
                            block_size=BLOCK_SIZE, head_dim=HEAD_DIM):
    """Workspace bytes of the grouped entry points: the split-K bound plus the
    partial slots of shared prefixes up to max_shared_tokens."""
    return int(lib().pkv_paged_attention_grouped_workspace_bytes(
        num_seqs, num_q_heads, max_blocks_per_seq, block_size, head_dim, max_shared_tokens))


def paged_attention_decode_grouped(out, q, k_cache, v_cache, block_tables, context_lens,
                                   group_first, seq_group, group_shared, max_shared_tokens,
                                   max_own_tokens, scale, workspace=None, dev_err=None,
                                   stream=None, prepare=False):
    """Same result as paged_attention_decode; each group's shared prefix is read
    once for all its members (see shared_prefix_groups).  prepare=True returns a
    PreparedLaunch instead of launching."""
    _dev(q, "q", torch.float16, 3)
    _dev(out, "out", torch.float16, 3)
    _dev(k_cache, "k_cache", torch.float16, 4)
    _dev(v_cache, "v_cache", torch.float16, 4)
    _dev(block_tables, "block_tables", torch.int32, 2)
    _dev(context_lens, "context_lens", torch.int32, 1)
    for name, t in (("group_first", group_first), ("seq_group", seq_group),
                    ("group_shared", group_shared)):
        _dev(t, name, torch.int32, 1)
    S, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    G = group_shared.shape[0]
    if group_first.shape[0] != G + 1 or seq_group.shape[0] != S:
        raise ValueError("group arrays do not match")
    max_blocks = block_tables.shape[1]
    need = grouped_workspace_bytes(S, Hq, max_blocks, int(max_shared_tokens), bs, D)
    if need and workspace is None:
        workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
            _ptr(context_lens), _ptr(group_first), _ptr(seq_group), _ptr(group_shared), G,
            int(max_shared_tokens), int(max_own_tokens), S, Hq, Hkv, D, bs, nb, max_blocks,
            float(scale), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream_handle(stream))
    keep = (out, q, k_cache, v_cache, block_tables, context_lens, group_first, seq_group,
            group_shared, workspace, dev_err, stream)
    return _issue(lib().pkv_paged_attention_decode_grouped, args,
                  "paged_attention_decode_grouped", keep, prepare, out)


def paged_attention_decode_grouped_fused(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                         context_lens, group_first, seq_group, group_shared,
                                         max_shared_tokens, max_own_tokens, scale,
                                         workspace=None, dev_err=None, stream=None,
                                         prepare=False, cow=None):
    """One launch: store k_new[s]/v_new[s] at position context_lens[s] - 1 of each
    sequence (a block past its group's shared prefix) and attend as
    paged_attention_decode_grouped.  cow=(cow_block, cow_src) also makes the
    copy-on-write copies in the same launch (see paged_attention_decode_fused)."""
    _dev(q, "q", torch.float16, 3)
    _dev(out, "out", torch.float16, 3)
    _dev(k_new, "k_new", torch.float16, 3)
    _dev(v_new, "v_new", torch.float16, 3)
    _dev(k_cache, "k_cache", torch.float16, 4)
    _dev(v_cache, "v_cache", torch.float16, 4)
    _dev(block_tables, "block_tables", torch.int32, 2)
    _dev(context_lens, "context_lens", torch.int32, 1)
    for name, t in (("group_first", group_first), ("seq_group", seq_group),
                    ("group_shared", group_shared)):
        _dev(t, name, torch.int32, 1)
    S, Hq, D = q.shape
    nb, bs, Hkv, _ = k_cache.shape
    if k_new.shape != (S, Hkv, D) or v_new.shape != k_new.shape:
        raise ValueError("k_new / v_new must be [num_seqs, num_kv_heads, head_dim]")
    G = group_shared.shape[0]
    if group_first.shape[0] != G + 1 or seq_group.shape[0] != S:
        raise ValueError("group arrays do not match")
    max_blocks = block_tables.shape[1]
    need = grouped_workspace_bytes(S, Hq, max_blocks, int(max_shared_tokens), bs, D)
    if need and workspace is None:
        workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if cow is not None:
        cb, cs = _cow_args(cow, S)
        args = (_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                _ptr(block_tables), _ptr(context_lens), _ptr(group_first), _ptr(seq_group),
                _ptr(group_shared), G, int(max_shared_tokens), int(max_own_tokens), _ptr(cb),
                _ptr(cs), S, Hq, Hkv, D, bs, nb, max_blocks, float(scale), _ptr(workspace),
                ws_bytes, _ptr(dev_err), _stream_handle(stream))
        keep = (out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, group_first,
                seq_group, group_shared, cb, cs, workspace, dev_err, stream)
        return _issue(lib().pkv_paged_attention_decode_grouped_fused_cow, args,
                      "paged_attention_decode_grouped_fused_cow", keep, prepare, out)
    args = (_ptr(out), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
            _ptr(block_tables), _ptr(context_lens), _ptr(group_first), _ptr(seq_group),
            _ptr(group_shared), G, int(max_shared_tokens), int(max_own_tokens), S, Hq, Hkv, D,
            bs, nb, max_blocks, float(scale), _ptr(workspace), ws_bytes, _ptr(dev_err),
            _stream_handle(stream))
    keep = (out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, group_first,
            seq_group, group_shared, workspace, dev_err, stream)
    return _issue(lib().pkv_paged_attention_decode_grouped_fused, args,
                  "paged_attention_decode_grouped_fused", keep, prepare, out)


# ---- prompt attention ------------------------------------------------------------------
# The checks of these entry points run once per call of a few microseconds: one
# expression that holds for good arguments, and only where it does not the checks
# that say what is wrong.

_F16, _F32, _I32 = torch.float16, torch.float32, torch.int32


def _explain(*specs):
    """Raise for the first (tensor, name, dtype, ndim) that is not as it should be."""
    for spec in specs:
        if _dev(*spec).get_device() != _get_device():
            raise ValueError("%s must be on the current CUDA device" % spec[1])
    raise ValueError("arguments do not fit together")


def _check_side(workspace, dev_err):
    """What the caller brings beside the data: a kernel writes it, so it is memory of the
    current device, without gaps (a gap is another tensor's), and the error word is int32."""
    dev = _get_device()
    if dev_err is not None:
        try:
            good = (dev_err.dtype is _I32 and dev_err.get_device() == dev and
                    dev_err.is_contiguous() and dev_err.numel() > 0)
        except (AttributeError, RuntimeError):
            good = False
        if not good:
            _explain((dev_err, "dev_err", _I32))
    if workspace is not None:
        try:
            good = workspace.get_device() == dev and workspace.is_contiguous()
        except (AttributeError, RuntimeError):
            good = False
        if not good:
            _explain((workspace, "workspace", getattr(workspace, "dtype", None)))


@functools.lru_cache(maxsize=256)
def prefill_workspace_bytes(num_tokens, num_seqs, num_q_heads, num_kv_heads, max_blocks_per_seq,
                            block_size=BLOCK_SIZE):
    """Bytes of partials paged_attention_prefill needs for these sizes (0 unless it
    splits the key axis)."""
    return int(lib().pkv_paged_attention_prefill_workspace_bytes(
        num_tokens, num_seqs, num_q_heads, num_kv_heads, max_blocks_per_seq, block_size))


def paged_attention_prefill(out, q, k_cache, v_cache, block_tables, context_lens, query_start,
                            scale, workspace=None, dev_err=None, stream=None, prepare=False):
    """Causal attention of packed prompt rows over the paged cache: sequence s owns rows
    query_start[s] .. query_start[s + 1] - 1 of q and out [T, Hq, 128], the last of its
    context_lens[s] tokens, all of whose K/V are in the cache.
    prepare=True returns a PreparedLaunch instead of launching."""
    try:
        dev = _get_device()
        good = (q.dtype is _F16 and q.get_device() == dev and q.is_contiguous() and
                out.dtype is _F16 and out.get_device() == dev and out.is_contiguous() and
                k_cache.dtype is _F16 and k_cache.get_device() == dev and
                k_cache.is_contiguous() and
                v_cache.dtype is _F16 and v_cache.get_device() == dev and
                v_cache.is_contiguous() and
                block_tables.dtype is _I32 and block_tables.get_device() == dev and
                block_tables.is_contiguous() and
                context_lens.dtype is _I32 and context_lens.get_device() == dev and
                context_lens.is_contiguous() and
                query_start.dtype is _I32 and query_start.get_device() == dev and
                query_start.is_contiguous()
                and q.dim() == 3 and k_cache.dim() == 4 and block_tables.dim() == 2)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        _explain((q, "q", _F16, 3), (out, "out", _F16, 3), (k_cache, "k_cache", _F16, 4),
                 (v_cache, "v_cache", _F16, 4), (block_tables, "block_tables", _I32, 2),
                 (context_lens, "context_lens", _I32, 1), (query_start, "query_start", _I32, 1))
    T, Hq, D = shape = q.shape
    nb, bs, Hkv, D2 = cache = k_cache.shape
    S, max_blocks = block_tables.shape
    if out.shape != shape or v_cache.shape != cache or D2 != D:
        raise ValueError("shape mismatch")
    if query_start.shape != (S + 1,) or context_lens.shape != (S,):
        raise ValueError("query_start must have num_seqs + 1 entries, context_lens num_seqs")
    if workspace is not None or dev_err is not None:
        _check_side(workspace, dev_err)
    if workspace is None:
        need = prefill_workspace_bytes(T, S, Hq, Hkv, max_blocks, bs)
        if need:
            workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            block_tables.data_ptr(), context_lens.data_ptr(), query_start.data_ptr(), T, S, Hq,
            Hkv, D, bs, nb, max_blocks, float(scale), _ptr(workspace), ws_bytes, _ptr(dev_err),
            _stream_handle(stream))
    keep = (out, q, k_cache, v_cache, block_tables, context_lens, query_start, workspace, dev_err,
            stream) if prepare else None
    return _run(lib().pkv_paged_attention_prefill, args, "paged_attention_prefill", prepare, keep,
                out)


def prompt_attention(out, q, k, v, query_start, scale, dev_err=None, stream=None, prepare=False):
    """Causal attention of whole packed prompts: q and out [T, Hq, 128], k and v [T, Hkv,
    128], sequence s owning rows query_start[s] .. query_start[s + 1] - 1 of each.
    prepare=True returns a PreparedLaunch instead of launching."""
    try:
        dev = _get_device()
        good = (q.dtype is _F16 and q.get_device() == dev and q.is_contiguous() and
                out.dtype is _F16 and out.get_device() == dev and out.is_contiguous() and
                k.dtype is _F16 and k.get_device() == dev and k.is_contiguous() and
                v.dtype is _F16 and v.get_device() == dev and v.is_contiguous() and
                query_start.dtype is _I32 and query_start.get_device() == dev and
                query_start.is_contiguous()
                and q.dim() == 3 and k.dim() == 3 and query_start.dim() == 1)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        _explain((q, "q", _F16, 3), (out, "out", _F16, 3), (k, "k", _F16, 3), (v, "v", _F16, 3),
                 (query_start, "query_start", _I32, 1))
    T, Hq, D = shape = q.shape
    T2, Hkv, D2 = rows = k.shape
    if out.shape != shape or T2 != T or D2 != D or v.shape != rows:
        raise ValueError("shape mismatch")
    S = query_start.shape[0] - 1
    if S < 0:
        raise ValueError("query_start must have num_seqs + 1 entries")
    if dev_err is not None:
        _check_side(None, dev_err)
    args = (out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), query_start.data_ptr(), T, S,
            Hq, Hkv, D, float(scale), _ptr(dev_err), _stream_handle(stream))
    keep = (out, q, k, v, query_start, dev_err, stream) if prepare else None
    return _run(lib().pkv_prompt_attention, args, "prompt_attention", prepare, keep, out)


# ---- 8-bit cache ----------------------------------------------------------------------

_CODES = {torch.int8: PKV_CODE_INT8, torch.float8_e4m3fn: PKV_CODE_E4M3}


def q8_cache(num_blocks, num_kv_heads, block_size=BLOCK_SIZE, dtype=torch.int8, device=None):
    """A zeroed 8-bit cache of one layer: (k_cache, v_cache, k_scale, v_scale), codes
    [num_blocks, block_size, num_kv_heads, 128] of ``dtype`` (torch.int8 or
    torch.float8_e4m3fn) and scales fp32 [num_blocks, stride], stride num_kv_heads
    rounded up to 4 (the columns past num_kv_heads are padding), which lets
    copy_blocks and swap_blocks move scales like codes."""
    if dtype not in _CODES:
        raise TypeError("an 8-bit cache is torch.int8 or torch.float8_e4m3fn, got %s" % dtype)
    dev = device or torch.cuda.current_device()
    shape = (num_blocks, block_size, num_kv_heads, HEAD_DIM)
    stride = -(-num_kv_heads // 4) * 4
    return tuple(torch.zeros(shape, dtype=torch.uint8, device=dev).view(dtype) for _ in "kv") + \
        tuple(torch.zeros((num_blocks, stride), dtype=torch.float32, device=dev) for _ in "kv")


def _q8_args(k_cache, v_cache, k_scale, v_scale):
    """The cache's code and sizes: code, num_blocks, block_size, Hkv, head_dim, stride."""
    try:
        dev = _get_device()
        code = _CODES.get(k_cache.dtype)
        good = (code is not None and k_cache.get_device() == dev and k_cache.is_contiguous() and
                v_cache.dtype is k_cache.dtype and v_cache.get_device() == dev and
                v_cache.is_contiguous() and
                k_scale.dtype is _F32 and k_scale.get_device() == dev and
                k_scale.is_contiguous() and
                v_scale.dtype is _F32 and v_scale.get_device() == dev and
                v_scale.is_contiguous() and
                k_cache.dim() == 4 and k_scale.dim() == 2)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        dtype = getattr(k_cache, "dtype", None)
        if dtype not in _CODES:
            raise TypeError("k_cache must be torch.int8 or torch.float8_e4m3fn, got %s" % dtype)
        _explain((k_cache, "k_cache", dtype, 4), (v_cache, "v_cache", dtype, 4),
                 (k_scale, "k_scale", _F32, 2), (v_scale, "v_scale", _F32, 2))
    nb, bs, Hkv, D = shape = k_cache.shape
    rows, stride = scales = k_scale.shape
    if v_cache.shape != shape or v_scale.shape != scales:
        raise ValueError("K and V caches, and their scales, must share one shape")
    if rows != nb or stride < Hkv:
        raise ValueError("scales must be [num_blocks, >= num_kv_heads]")
    return code, nb, bs, Hkv, D, stride


def reshape_and_cache_q8(k, v, query_start, block_tables, context_lens, k_cache, v_cache, k_scale,
                         v_scale, dev_err=None, stream=None, prepare=False):
    """Code the packed rows k, v [T, Hkv, 128] into an 8-bit cache: sequence s brings
    rows query_start[s] .. query_start[s + 1] - 1, the last of its context_lens[s]
    tokens.  One scale per (block, KV head): the largest magnitude over 127 (int8) or
    448 (e4m3); rows a block already holds are coded anew when its scale grows.
    prepare=True returns a PreparedLaunch instead of launching."""
    try:
        dev = _get_device()
        good = (k.dtype is _F16 and k.get_device() == dev and k.is_contiguous() and
                v.dtype is _F16 and v.get_device() == dev and v.is_contiguous() and
                query_start.dtype is _I32 and query_start.get_device() == dev and
                query_start.is_contiguous() and
                block_tables.dtype is _I32 and block_tables.get_device() == dev and
                block_tables.is_contiguous() and
                context_lens.dtype is _I32 and context_lens.get_device() == dev and
                context_lens.is_contiguous() and k.dim() == 3 and block_tables.dim() == 2)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        _explain((k, "k", _F16, 3), (v, "v", _F16, 3), (query_start, "query_start", _I32, 1),
                 (block_tables, "block_tables", _I32, 2), (context_lens, "context_lens", _I32, 1))
    code, nb, bs, Hkv, D, stride = _q8_args(k_cache, v_cache, k_scale, v_scale)
    T, Hkv2, D2 = rows = k.shape
    S, max_blocks = block_tables.shape
    if Hkv2 != Hkv or D2 != D or v.shape != rows:
        raise ValueError("shape mismatch")
    if query_start.shape != (S + 1,) or context_lens.shape != (S,):
        raise ValueError("query_start must have num_seqs + 1 entries, context_lens num_seqs")
    if dev_err is not None:
        _check_side(None, dev_err)
    args = (k.data_ptr(), v.data_ptr(), query_start.data_ptr(), block_tables.data_ptr(),
            context_lens.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), code, T, S, Hkv, D, bs, nb, max_blocks, stride, _ptr(dev_err),
            _stream_handle(stream))
    keep = (k, v, query_start, block_tables, context_lens, k_cache, v_cache, k_scale, v_scale,
            dev_err, stream) if prepare else None
    return _run(lib().pkv_reshape_and_cache_q8, args, "reshape_and_cache_q8", prepare, keep, None)


def paged_attention_decode_q8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                              context_lens, scale, workspace=None, dev_err=None, stream=None,
                              prepare=False):
    """paged_attention_decode over an 8-bit cache (see q8_cache, reshape_and_cache_q8);
    same workspace.  prepare=True returns a PreparedLaunch instead of launching."""
    try:
        dev = _get_device()
        good = (q.dtype is _F16 and q.get_device() == dev and q.is_contiguous() and
                out.dtype is _F16 and out.get_device() == dev and out.is_contiguous() and
                block_tables.dtype is _I32 and block_tables.get_device() == dev and
                block_tables.is_contiguous() and
                context_lens.dtype is _I32 and context_lens.get_device() == dev and
                context_lens.is_contiguous() and q.dim() == 3 and block_tables.dim() == 2)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        _explain((q, "q", _F16, 3), (out, "out", _F16, 3),
                 (block_tables, "block_tables", _I32, 2), (context_lens, "context_lens", _I32, 1))
    code, nb, bs, Hkv, D, stride = _q8_args(k_cache, v_cache, k_scale, v_scale)
    S, Hq, D2 = shape = q.shape
    if out.shape != shape or D2 != D:
        raise ValueError("shape mismatch")
    rows, max_blocks = block_tables.shape
    if rows != S or context_lens.shape != (S,):
        raise ValueError("block_tables / context_lens must have num_seqs rows")
    if workspace is not None or dev_err is not None:
        _check_side(workspace, dev_err)
    if workspace is None:
        need = workspace_bytes(S, Hq, max_blocks, bs)
        if need:
            workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), code, block_tables.data_ptr(),
            context_lens.data_ptr(), S, Hq, Hkv, D, bs, nb, max_blocks, stride, float(scale),
            _ptr(workspace), ws_bytes, _ptr(dev_err), _stream_handle(stream))
    keep = (out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, workspace,
            dev_err, stream) if prepare else None
    return _run(lib().pkv_paged_attention_decode_q8, args, "paged_attention_decode_q8", prepare,
                keep, out)


@functools.lru_cache(maxsize=256)
def prefill_q8_workspace_bytes(num_tokens, num_seqs, num_q_heads, num_kv_heads, max_blocks_per_seq,
                               block_size=BLOCK_SIZE):
    """Bytes of partials paged_attention_prefill_q8 needs for these sizes (0 unless it
    splits the key axis)."""
    return int(lib().pkv_paged_attention_prefill_q8_workspace_bytes(
        num_tokens, num_seqs, num_q_heads, num_kv_heads, max_blocks_per_seq, block_size))


def paged_attention_prefill_q8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables,
                               context_lens, query_start, scale, workspace=None, dev_err=None,
                               stream=None, prepare=False):
    """paged_attention_prefill over an 8-bit cache (see q8_cache, reshape_and_cache_q8,
    rope_and_cache_q8); workspace: prefill_q8_workspace_bytes.
    prepare=True returns a PreparedLaunch instead of launching."""
    try:
        dev = _get_device()
        good = (q.dtype is _F16 and q.get_device() == dev and q.is_contiguous() and
                out.dtype is _F16 and out.get_device() == dev and out.is_contiguous() and
                block_tables.dtype is _I32 and block_tables.get_device() == dev and
                block_tables.is_contiguous() and
                context_lens.dtype is _I32 and context_lens.get_device() == dev and
                context_lens.is_contiguous() and
                query_start.dtype is _I32 and query_start.get_device() == dev and
                query_start.is_contiguous() and q.dim() == 3 and block_tables.dim() == 2)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        _explain((q, "q", _F16, 3), (out, "out", _F16, 3),
                 (block_tables, "block_tables", _I32, 2), (context_lens, "context_lens", _I32, 1),
                 (query_start, "query_start", _I32, 1))
    code, nb, bs, Hkv, D, stride = _q8_args(k_cache, v_cache, k_scale, v_scale)
    T, Hq, D2 = shape = q.shape
    S, max_blocks = block_tables.shape
    if out.shape != shape or D2 != D:
        raise ValueError("shape mismatch")
    if query_start.shape != (S + 1,) or context_lens.shape != (S,):
        raise ValueError("query_start must have num_seqs + 1 entries, context_lens num_seqs")
    if workspace is not None or dev_err is not None:
        _check_side(workspace, dev_err)
    if workspace is None:
        need = prefill_q8_workspace_bytes(T, S, Hq, Hkv, max_blocks, bs)
        if need:
            workspace = _new_workspace(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = (out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            k_scale.data_ptr(), v_scale.data_ptr(), code, block_tables.data_ptr(),
            context_lens.data_ptr(), query_start.data_ptr(), T, S, Hq, Hkv, D, bs, nb, max_blocks,
            stride, float(scale), _ptr(workspace), ws_bytes, _ptr(dev_err), _stream_handle(stream))
    keep = (out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_start,
            workspace, dev_err, stream) if prepare else None
    return _run(lib().pkv_paged_attention_prefill_q8, args, "paged_attention_prefill_q8", prepare,
                keep, out)


# ---- rotary positions -------------------------------------------------------------------

def rope_table(inv_freq, num_positions, magnitude=1.0, device=None):
    """The table the rotary calls read: fp32 [num_positions, n, 2], magnitude times cosine
    and sine of position * inv_freq[j], the angles in 64 bits (at a million positions
    32 bits would be off by 0.03).  inv_freq: n radians a position, a sequence or a tensor."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device=dev)
    if f.dim() != 1 or num_positions <= 0:
        raise ValueError("need inv_freq [n] and a positive number of positions")
    table = torch.empty((num_positions, f.shape[0], 2), dtype=torch.float32, device=dev)
    for lo in range(0, num_positions, 1 << 16):   # a bounded amount of 64-bit intermediates
        hi = min(num_positions, lo + (1 << 16))
        angle = torch.arange(lo, hi, dtype=torch.float64, device=dev)[:, None] * f
        table[lo:hi, :, 0] = angle.cos() * magnitude
        table[lo:hi, :, 1] = angle.sin() * magnitude
    return table


def rope_sections(sizes, round_robin=False):
    """The axis of each pair for the rotary calls' ``axes``: sizes[a] pairs of axis a, one
    axis after the other, or dealt one to each axis in turn while it has some left."""
    if not round_robin:
        return tuple(a for a, m in enumerate(sizes) for _ in range(m))
    return tuple(a for r in range(max(sizes)) for a, m in enumerate(sizes) if r < m)


@functools.lru_cache(maxsize=256)
def _pack_axes(axes, n, num_axes):
    if len(axes) != n or not all(isinstance(a, int) and 0 <= a < num_axes for a in axes):
        raise ValueError("axes must be %d axis numbers below %d, one for each pair" % (n, num_axes))
    return bytes(axes)


def _rows_of(t, name, dev):
    """(tokens, heads, halves between tokens) of fp16 [T, H, 128] whose heads are contiguous;
    the tokens may lie further apart, as in a slice of a projection's output."""
    try:
        good = t.dtype is _F16 and t.get_device() == dev and t.dim() == 3
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("%s must be a CUDA tensor" % name)
        if t.dtype != _F16:
            raise TypeError("%s must be %s, got %s" % (name, _F16, t.dtype))
        if t.dim() != 3:
            raise ValueError("%s must have 3 dims, got %s" % (name, tuple(t.shape)))
        raise ValueError("%s must be on the current CUDA device" % name)
    T, H, D = t.shape
    a, b, c = t.stride()
    if D != HEAD_DIM or (c != 1 and T and H) or (b != HEAD_DIM and H > 1 and T):
        raise ValueError("%s must be [T, heads, %d] with each token's heads contiguous" %
                         (name, HEAD_DIM))
    if T <= 1:
        a = H * HEAD_DIM
    elif a & 7:
        raise ValueError("%s must have a multiple of 8 elements between tokens" % name)
    return T, H, a


def _rope_args(table, positions, axes, T, dev, required):
    """(positions, num_axes, axes, table, table rows, rot_dim) as the C calls take them."""
    try:
        rows, n, two = table.shape
        good = (table.dtype is _F32 and table.get_device() == dev and table.is_contiguous())
    except (AttributeError, RuntimeError, ValueError):
        good = False
    if not good:
        _explain((table, "table", _F32, 3))
    if two != 2:
        raise ValueError("table must be [positions, pairs, 2]")
    if positions is None:
        if required:
            raise TypeError("positions must be a CUDA tensor")
        if axes is None:
            return None, 1, None, table.data_ptr(), rows, 2 * n
        return None, 4, _pack_axes(tuple(axes), n, 4), table.data_ptr(), rows, 2 * n
    try:
        good = (positions.dtype is _I32 and positions.get_device() == dev and
                positions.is_contiguous())
        shape = positions.shape
    except (AttributeError, RuntimeError):
        good = False
    if not good or not 1 <= len(shape) <= 2:
        _explain((positions, "positions", _I32, 2 if getattr(positions, "ndim", 1) > 1 else 1))
    if shape[-1] != T:
        raise ValueError("positions must have one entry for each token")
    num = shape[0] if len(shape) == 2 else 1
    if not 1 <= num <= 4:
        raise ValueError("positions must have 1 to 4 axes")
    if axes is not None:
        axes = _pack_axes(tuple(axes), n, num)
    elif num > 1:
        raise ValueError("axes must say which of the %d axes each pair follows" % num)
    return positions.data_ptr(), num, axes, table.data_ptr(), rows, 2 * n


def _check_out_stride(name, T, H, stride):
    if T > 1 and stride < H * HEAD_DIM:
        raise ValueError("tokens of %s overlap" % name)


def rotary_embedding(q_out, k_out, q, k, positions, table, axes=None, adjacent=False, dev_err=None,
                     stream=None, prepare=False):
    """q_out = q and k_out = k [T, heads, 128] rotated by ``positions`` int32 [T], or [axes, T]
    with ``axes`` the axis of each pair (rope_sections), through ``table`` (rope_table).
    Pairs are dims (j, j + n), or (2j, 2j + 1) if ``adjacent``.  The tensors may be slices
    of a projection's output, and q_out q, k_out k (in place); k and k_out may be None.
    prepare=True returns a PreparedLaunch instead of launching."""
    dev = _get_device()
    try:
        T, Hq, D = shape = q.shape
        Tk, Hkv, Dk = shape_k = k.shape
        (so, a, b), (sq, c, d) = q_out.stride(), q.stride()
        (sko, e, f), (sk, g, h) = k_out.stride(), k.stride()
        good = (q.dtype is _F16 and q_out.dtype is _F16 and k.dtype is _F16 and
                k_out.dtype is _F16 and q.get_device() == dev and q_out.get_device() == dev and
                k.get_device() == dev and k_out.get_device() == dev and
                q_out.shape == shape and k_out.shape == shape_k and Tk == T and
                D == Dk == a == c == e == g == 128 and b == d == f == h == 1 and
                not (so | sq | sko | sk) & 7)
    except (AttributeError, RuntimeError, ValueError):
        good = False
    if not good:      # what is wrong, or a shape of one token or head with other strides
        T, Hq, sq = _rows_of(q, "q", dev)
        To, Ho, so = _rows_of(q_out, "q_out", dev)
        Hkv = sk = sko = 0
        if (k is None) != (k_out is None):
            raise TypeError("k and k_out go together")
        if k is not None:
            Tk, Hkv, sk = _rows_of(k, "k", dev)
            Tko, Hko, sko = _rows_of(k_out, "k_out", dev)
            if Tk != T or Tko != T or Hko != Hkv:
                raise ValueError("shape mismatch")
        if To != T or Ho != Hq:
            raise ValueError("shape mismatch")
    _check_out_stride("q_out", T, Hq, so)
    _check_out_stride("k_out", T, Hkv, sko)
    rot = _rope_args(table, positions, axes, T, dev, True)
    if dev_err is not None:
        _check_side(None, dev_err)
    args = (q_out.data_ptr(), _ptr(k_out), q.data_ptr(), _ptr(k), so, sko, sq, sk, *rot,
            1 if adjacent else 0, T, Hq, Hkv, HEAD_DIM, _ptr(dev_err), _stream_handle(stream))
    keep = (q_out, k_out, q, k, positions, table, dev_err, stream) if prepare else None
    return _run(lib().pkv_rotary_embedding, args, "rotary_embedding", prepare, keep, None)


def _append_args(q_out, q, k, v, query_start, block_tables, context_lens, table, positions, axes):
    """What both caches' calls share: sizes (T, S, Hq, Hkv, max_blocks), strides, rotation."""
    dev = _get_device()
    try:
        T, Hq, D = shape = q.shape
        Tk, Hkv, Dk = shape_k = k.shape
        S, max_blocks = block_tables.shape
        (so, a, b), (sq, c, d) = q_out.stride(), q.stride()
        (sk, e, f), (sv, g, h) = k.stride(), v.stride()
        good = (q.dtype is _F16 and q_out.dtype is _F16 and k.dtype is _F16 and v.dtype is _F16 and
                q.get_device() == dev and q_out.get_device() == dev and k.get_device() == dev and
                v.get_device() == dev and q_out.shape == shape and v.shape == shape_k and
                Tk == T and D == Dk == a == c == e == g == 128 and b == d == f == h == 1 and
                not (so | sq | sk | sv) & 7 and
                query_start.dtype is _I32 and query_start.get_device() == dev and
                query_start.is_contiguous() and
                block_tables.dtype is _I32 and block_tables.get_device() == dev and
                block_tables.is_contiguous() and
                context_lens.dtype is _I32 and context_lens.get_device() == dev and
                context_lens.is_contiguous())
    except (AttributeError, RuntimeError, ValueError, TypeError):
        good = False
    if not good:      # what is wrong, or a shape of one token or head with other strides
        T, Hq, sq = _rows_of(q, "q", dev)
        To, Ho, so = _rows_of(q_out, "q_out", dev)
        Tk, Hkv, sk = _rows_of(k, "k", dev)
        Tv, Hv, sv = _rows_of(v, "v", dev)
        for t, name, dim in ((query_start, "query_start", 1), (block_tables, "block_tables", 2),
                             (context_lens, "context_lens", 1)):
            if _dev(t, name, _I32, dim).get_device() != dev:
                raise ValueError("%s must be on the current CUDA device" % name)
        if To != T or Tk != T or Tv != T or Ho != Hq or Hv != Hkv:
            raise ValueError("shape mismatch")
        S, max_blocks = block_tables.shape
    if query_start.shape != (S + 1,) or context_lens.shape != (S,):
        raise ValueError("query_start must have num_seqs + 1 entries, context_lens num_seqs")
    _check_out_stride("q_out", T, Hq, so)
    return (T, S, Hq, Hkv, max_blocks), (so, sq, sk, sv), \
        _rope_args(table, positions, axes, T, dev, False)


def rope_and_cache(q_out, q, k, v, query_start, block_tables, context_lens, k_cache, v_cache, table,
                   positions=None, axes=None, adjacent=False, dev_err=None, stream=None,
                   prepare=False):
    """One launch: q [T, Hq, 128] rotated into q_out, k rotated and v as it is written to the
    paged fp16 cache.  Sequence s brings rows query_start[s] .. query_start[s + 1] - 1, the
    last of its context_lens[s] tokens; without ``positions`` a token's position is its place
    in the sequence.  ``table``, ``positions``, ``axes``, ``adjacent`` and the layout of q, k,
    v and q_out as in rotary_embedding.
    prepare=True returns a PreparedLaunch instead of launching."""
    (T, S, Hq, Hkv, max_blocks), strides, rot = _append_args(
        q_out, q, k, v, query_start, block_tables, context_lens, table, positions, axes)
    try:
        dev = _get_device()
        good = (k_cache.dtype is _F16 and k_cache.get_device() == dev and
                k_cache.is_contiguous() and
                v_cache.dtype is _F16 and v_cache.get_device() == dev and
                v_cache.is_contiguous() and k_cache.dim() == 4)
    except (AttributeError, RuntimeError):
        good = False
    if not good:
        _explain((k_cache, "k_cache", _F16, 4), (v_cache, "v_cache", _F16, 4))
    nb, bs, Hc, D = cache = k_cache.shape
    if v_cache.shape != cache or Hc != Hkv or D != HEAD_DIM:
        raise ValueError("shape mismatch")
    if dev_err is not None:
        _check_side(None, dev_err)
    args = (q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides,
            query_start.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), *rot, 1 if adjacent else 0, T, S, Hq, Hkv, D,
            bs, nb, max_blocks, _ptr(dev_err), _stream_handle(stream))
    keep = (q_out, q, k, v, query_start, block_tables, context_lens, k_cache, v_cache, table,
            positions, dev_err, stream) if prepare else None
    return _run(lib().pkv_rope_and_cache, args, "rope_and_cache", prepare, keep, None)


def rope_and_cache_q8(q_out, q, k, v, query_start, block_tables, context_lens, k_cache, v_cache,
                      k_scale, v_scale, table, positions=None, axes=None, adjacent=False,
                      dev_err=None, stream=None, prepare=False):
    """rope_and_cache into an 8-bit cache (q8_cache): the rule of reshape_and_cache_q8 on the
    rotated k in 32 bits and on v.
    prepare=True returns a PreparedLaunch instead of launching."""
    (T, S, Hq, Hkv, max_blocks), strides, rot = _append_args(
        q_out, q, k, v, query_start, block_tables, context_lens, table, positions, axes)
    code, nb, bs, Hc, D, stride = _q8_args(k_cache, v_cache, k_scale, v_scale)
    if Hc != Hkv or D != HEAD_DIM:
        raise ValueError("shape mismatch")
    if dev_err is not None:
        _check_side(None, dev_err)
    args = (q_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides,
            query_start.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), code,
            *rot, 1 if adjacent else 0, T, S, Hq, Hkv, D, bs, nb, max_blocks, stride,
            _ptr(dev_err), _stream_handle(stream))
    keep = (q_out, q, k, v, query_start, block_tables, context_lens, k_cache, v_cache, k_scale,
            v_scale, table, positions, dev_err, stream) if prepare else None
    return _run(lib().pkv_rope_and_cache_q8, args, "rope_and_cache_q8", prepare, keep, None)
