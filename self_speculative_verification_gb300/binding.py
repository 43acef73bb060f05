"""Python binding of the libspecverify C ABI (argument marshalling only).

Every function here has the name of the C entry point it calls, checks the
tensors it is handed (CUDA device, dtype, contiguity, shape), passes raw
device pointers plus the current torch CUDA stream, and raises
``SpecError`` on any non-zero return code.  No arithmetic of the
verification step happens in Python: if the shared library is missing,
``load_library`` raises and nothing runs.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int, c_longlong, c_size_t, c_void_p

import torch

from . import _build

# return codes / enums (include/specverify.h)
SPEC_OK = 0
SPEC_ERR_INVALID_ARG = 1
SPEC_ERR_UNSUPPORTED = 2
SPEC_ERR_CAPACITY = 4
SPEC_ERR_CUDA = 5
SPEC_ERR_DEVICE = 6
SPEC_F32 = 0
SPEC_BF16 = 1
SPEC_KV_CONTIGUOUS = 0
SPEC_KV_PAGED = 1
SPEC_ACCEPT_THRESH_CHAIN = 0
SPEC_ACCEPT_GREEDY_TREE = 1
SPEC_ROW_VALID = 1
SPEC_ROW_SEES_SOFT = 2
SPEC_ROPE_PAIRS = 0
SPEC_ROPE_HALVES = 1
SPEC_ROPE_PLAIN = 0
SPEC_ROPE_LINEAR = 1
SPEC_ROPE_RAMP = 2
SPEC_DEV_BAD_TREE = 0x01
SPEC_DEV_BAD_PAGE = 0x02
SPEC_DEV_SEQ_OVERFLOW = 0x04
SPEC_DEV_CAPACITY = 0x08
SPEC_DEV_BAD_INDEX = 0x10
SPEC_DEV_TIMEOUT = 0x20

EXPORTS = ("spec_version", "spec_status_string", "spec_mask_build",
           "spec_verify_attn_workspace_size", "spec_verify_attn",
           "spec_verify_attn_noalloc", "spec_vocab_reduce", "spec_accept", "kv_commit",
           "spec_get_status", "spec_la_prefill_attn", "spec_accept_soft", "spec_draft_tree",
           "spec_prune_tree", "spec_stream_rotate_values", "spec_future_gather",
           "spec_set_wait_limit", "spec_verify_attn_kv8_workspace_size", "spec_verify_attn_kv8",
           "kv8_commit", "kv8_append", "spec_page_plan", "spec_logits_adjust", "spec_rope_freqs",
           "spec_rope", "kv_append", "spec_chunk_attn_workspace_size", "spec_chunk_attn",
           "spec_chunk_attn_kv8_workspace_size", "spec_chunk_attn_kv8")
SPEC_NOALLOC_SCRATCH_BYTES = 64 << 20


class SpecError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} failed: {msg} (code {code})")
        self.code = code


class KvDesc(ctypes.Structure):
    _fields_ = [("kind", c_int), ("dtype", c_int), ("n_kv_heads", c_int),
                ("head_dim", c_int), ("k", c_void_p), ("v", c_void_p),
                ("batch", c_int), ("max_seq", c_int), ("n_pages", c_int),
                ("page_size", c_int), ("max_pages_per_seq", c_int),
                ("page_table", c_void_p)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_rows", c_int), ("n_q_heads", c_int),
                ("n_kv_heads", c_int), ("head_dim", c_int), ("dtype", c_int),
                ("n_soft", c_int), ("scale", c_float), ("split_tokens", c_int)]


class AcceptDesc(ctypes.Structure):
    _fields_ = [("mode", c_int), ("tau", c_float), ("batch", c_int),
                ("n_judge_rows", c_int), ("vocab", c_int), ("logit_dtype", c_int),
                ("max_nodes", c_int), ("path_cap", c_int)]


class SoftDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_judge_rows", c_int), ("n_draft_rows", c_int),
                ("vocab", c_int), ("logit_dtype", c_int), ("max_nodes", c_int),
                ("path_cap", c_int), ("temperature", c_float)]


class DraftDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_stream_rows", c_int), ("gamma", c_int), ("k", c_int),
                ("vocab", c_int), ("logit_dtype", c_int), ("max_nodes", c_int),
                ("vparent_rows", c_int)]


class PruneDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("max_nodes", c_int), ("vocab", c_int),
                ("logit_dtype", c_int), ("threshold", c_float), ("gamma", c_int),
                ("vparent_rows", c_int)]


class RotateDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_rows", c_int), ("n_kv_heads", c_int),
                ("head_dim", c_int), ("dtype", c_int), ("gamma", c_int), ("eps", c_float)]


class PrefillDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_orig", c_int), ("n_look", c_int),
                ("n_q_heads", c_int), ("n_kv_heads", c_int), ("head_dim", c_int),
                ("dtype", c_int), ("scale", c_float)]


class Kv8Desc(ctypes.Structure):
    _fields_ = [("n_kv_heads", c_int), ("head_dim", c_int), ("kv", c_void_p),
                ("scales", c_void_p), ("batch", c_int), ("n_pages", c_int),
                ("page_size", c_int), ("max_pages_per_seq", c_int), ("page_table", c_void_p)]


class LogitsDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_judge_rows", c_int), ("vocab", c_int),
                ("logit_dtype", c_int), ("max_nodes", c_int), ("hist_cap", c_int),
                ("n_bias", c_int), ("n_masks", c_int)]


class ChunkDesc(ctypes.Structure):
    _fields_ = [("batch", c_int), ("n_tokens", c_int), ("n_q_heads", c_int),
                ("n_kv_heads", c_int), ("head_dim", c_int), ("dtype", c_int), ("scale", c_float)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("n_tokens", c_int), ("n_q_heads", c_int), ("n_k_heads", c_int),
                ("head_dim", c_int), ("rot_dim", c_int), ("layout", c_int), ("dtype", c_int),
                ("attention", c_float)]


_lib = None


def library_path() -> str:
    return os.environ.get("SPECVERIFY_LIB", _build.LIB)


def load_library():
    """Load libspecverify.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libspecverify is not built ({path} missing); "
                           "run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    vp = c_void_p
    sig = {
        "spec_version": ([], c_int),
        "spec_status_string": ([c_int], ctypes.c_char_p),
        "spec_mask_build": ([vp, vp, c_int, c_int, vp, vp, vp], c_int),
        "spec_verify_attn_workspace_size": ([POINTER(AttnDesc), POINTER(KvDesc),
                                             POINTER(c_size_t)], c_int),
        "spec_verify_attn": ([POINTER(AttnDesc), vp, POINTER(KvDesc), vp, vp, vp, vp,
                              vp, vp, vp, vp, vp, vp, c_size_t, vp], c_int),
        "spec_verify_attn_noalloc": ([POINTER(AttnDesc), vp, POINTER(KvDesc), vp, vp, vp, vp,
                                      vp, vp, vp, vp, vp, vp], c_int),
        "spec_vocab_reduce": ([vp, c_int, c_int, c_int, vp, vp, vp, vp, vp], c_int),
        "spec_accept": ([POINTER(AcceptDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                         vp, vp, vp], c_int),
        "kv_commit": ([POINTER(KvDesc), c_int, c_int, vp, vp, c_int, vp, vp, vp, vp,
                       c_int, vp, vp], c_int),
        "spec_get_status": ([vp, POINTER(ctypes.c_int32)], c_int),
        "spec_set_wait_limit": ([ctypes.c_longlong], ctypes.c_longlong),
        "spec_la_prefill_attn": ([POINTER(PrefillDesc), vp, vp, vp, vp, vp, vp], c_int),
        "spec_accept_soft": ([POINTER(SoftDesc)] + [vp] * 16, c_int),
        "spec_draft_tree": ([POINTER(DraftDesc)] + [vp] * 8, c_int),
        "spec_prune_tree": ([POINTER(PruneDesc)] + [vp] * 10, c_int),
        "spec_stream_rotate_values": ([POINTER(RotateDesc), vp, vp, vp], c_int),
        "spec_future_gather": ([c_int, c_int, c_int, c_int, vp, vp, c_int, vp, vp], c_int),
        "spec_verify_attn_kv8_workspace_size": ([POINTER(AttnDesc), POINTER(Kv8Desc),
                                                 POINTER(c_size_t)], c_int),
        "spec_verify_attn_kv8": ([POINTER(AttnDesc), vp, POINTER(Kv8Desc)] + [vp] * 10 +
                                 [c_size_t, vp], c_int),
        "kv8_commit": ([POINTER(Kv8Desc), c_int, c_int, c_int, vp, vp, c_int, vp, vp, vp, vp, c_int,
                        vp, vp], c_int),
        "kv8_append": ([POINTER(Kv8Desc), c_int, c_int, vp, c_longlong, vp, c_longlong, vp, vp],
                       c_int),
        "spec_page_plan": ([c_int, c_int, c_int, c_int, vp, vp, vp, vp, c_int, vp, vp, c_longlong,
                            vp, vp, vp], c_int),
        "spec_logits_adjust": ([POINTER(LogitsDesc)] + [vp] * 16, c_int),
        "spec_rope_freqs": ([c_int, c_double, c_int] + [c_double] * 4 + [POINTER(c_double)], c_int),
        "spec_rope": ([POINTER(RopeDesc), POINTER(c_double)] + [vp, c_longlong] * 4 +
                      [vp, c_int, vp, vp, vp], c_int),
        "kv_append": ([POINTER(KvDesc), c_int, vp, c_longlong, vp, c_longlong, vp, vp], c_int),
        "spec_chunk_attn_workspace_size": ([POINTER(ChunkDesc), POINTER(KvDesc),
                                            POINTER(c_size_t)], c_int),
        "spec_chunk_attn": ([POINTER(ChunkDesc), vp, c_longlong, POINTER(KvDesc)] + [vp] * 5 +
                            [c_size_t, vp], c_int),
        "spec_chunk_attn_kv8_workspace_size": ([POINTER(ChunkDesc), POINTER(Kv8Desc),
                                                POINTER(c_size_t)], c_int),
        "spec_chunk_attn_kv8": ([POINTER(ChunkDesc), vp, c_longlong, POINTER(Kv8Desc)] + [vp] * 5 +
                                [c_size_t, vp], c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _check(fn, code):
    if code != SPEC_OK:
        msg = load_library().spec_status_string(code).decode()
        raise SpecError(fn, code, msg)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return c_void_p(t.data_ptr())


def spec_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ----------------------------------------------------------------- descriptors

def kv_desc_contiguous(k: torch.Tensor, v: torch.Tensor) -> KvDesc:
    """k, v: [B][Hkv][max_seq][d]."""
    if k.shape != v.shape or k.dim() != 4:
        raise ValueError("k and v must be [B][Hkv][max_seq][d]")
    _ptr(k, name="k"), _ptr(v, k.dtype, "v")
    B, Hkv, S, d = k.shape
    desc = KvDesc(SPEC_KV_CONTIGUOUS, spec_dtype(k), Hkv, d, k.data_ptr(), v.data_ptr(),
                  B, S, 0, 0, 0, None)
    desc.device = k.get_device()
    return desc


def kv_desc_paged(k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor) -> KvDesc:
    """k, v: [n_pages][Hkv][d / 64][page_size][64]; page_table int32 [B][max_pages]."""
    if k.shape != v.shape or k.dim() != 5 or k.shape[4] != 64:
        raise ValueError("k and v must be [n_pages][Hkv][d / 64][page_size][64]")
    _ptr(k, name="k"), _ptr(v, k.dtype, "v")
    _ptr(page_table, torch.int32, "page_table")
    P, Hkv, nblk, ps, _ = k.shape
    d = nblk * 64
    B, maxp = page_table.shape
    desc = KvDesc(SPEC_KV_PAGED, spec_dtype(k), Hkv, d, k.data_ptr(), v.data_ptr(),
                  B, 0, P, ps, maxp, page_table.data_ptr())
    desc.device = k.get_device()
    return desc


def attn_desc(batch, n_rows, n_q_heads, n_kv_heads, head_dim, dtype, n_soft=0,
              scale=0.0, split_tokens=0) -> AttnDesc:
    return AttnDesc(batch, n_rows, n_q_heads, n_kv_heads, head_dim, dtype, n_soft,
                    scale, split_tokens)


def accept_desc(mode, tau, batch, n_judge_rows, vocab, logit_dtype, max_nodes,
                path_cap) -> AcceptDesc:
    return AcceptDesc(mode, tau, batch, n_judge_rows, vocab, logit_dtype, max_nodes,
                      path_cap)


# ------------------------------------------------------------------- entry points

def prefill_desc(batch, n_orig, n_look, n_q_heads, n_kv_heads, head_dim, dtype=SPEC_BF16,
                 scale=0.0) -> PrefillDesc:
    return PrefillDesc(batch, n_orig, n_look, n_q_heads, n_kv_heads, head_dim, dtype, scale)


def soft_desc(batch, n_judge_rows, n_draft_rows, vocab, logit_dtype, max_nodes, path_cap,
              temperature=1.0) -> SoftDesc:
    return SoftDesc(batch, n_judge_rows, n_draft_rows, vocab, logit_dtype, max_nodes, path_cap,
                    temperature)


def spec_version() -> int:
    return load_library().spec_version()


def spec_mask_build(vparent, soft_flags, vis, row_flags, stream=None):
    lib = load_library()
    B, R = vparent.shape
    W = (R + 31) // 32
    if tuple(vis.shape) != (B, R, W) or tuple(row_flags.shape) != (B, R):
        raise ValueError("vis must be [B][R][ceil(R/32)], row_flags [B][R]")
    _check("spec_mask_build", lib.spec_mask_build(
        _ptr(vparent, torch.int32, "vparent"), _ptr(soft_flags, torch.uint8, "soft_flags"),
        B, R, _ptr(vis, torch.int32, "vis"), _ptr(row_flags, torch.uint8, "row_flags"),
        _stream(stream)))


def spec_verify_attn_workspace_size(attn: AttnDesc, cache: KvDesc) -> int:
    lib = load_library()
    n = c_size_t(0)
    _check("spec_verify_attn_workspace_size",
           lib.spec_verify_attn_workspace_size(ctypes.byref(attn), ctypes.byref(cache),
                                               ctypes.byref(n)))
    return n.value


def spec_verify_attn(attn: AttnDesc, q, cache: KvDesc, kb, vb, soft_k, soft_v, seq_len,
                     vis, row_flags, o, lse, workspace, stream=None):
    lib = load_library()
    dt = q.dtype
    for name, t in (("kb", kb), ("vb", vb), ("o", o)):
        _ptr(t, dt, name)
    _check("spec_verify_attn", lib.spec_verify_attn(
        ctypes.byref(attn), _ptr(q, name="q"), ctypes.byref(cache), _ptr(kb), _ptr(vb),
        _ptr(soft_k, dt, "soft_k"), _ptr(soft_v, dt, "soft_v"),
        _ptr(seq_len, torch.int32, "seq_len"), _ptr(vis, torch.int32, "vis"),
        _ptr(row_flags, torch.uint8, "row_flags"), _ptr(o), _ptr(lse, torch.float32, "lse"),
        _ptr(workspace, name="workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def spec_verify_attn_noalloc(attn: AttnDesc, q, cache: KvDesc, kb, vb, soft_k, soft_v,
                             seq_len, vis, row_flags, o, lse, stream=None):
    """spec_verify_attn without a workspace: for callers that cannot
    allocate device memory; the library's own fixed scratch array is used
    (shared by all calls on a device, so overlapping calls must not run)."""
    lib = load_library()
    dt = q.dtype
    for name, t in (("kb", kb), ("vb", vb), ("o", o)):
        _ptr(t, dt, name)
    _check("spec_verify_attn_noalloc", lib.spec_verify_attn_noalloc(
        ctypes.byref(attn), _ptr(q, name="q"), ctypes.byref(cache), _ptr(kb), _ptr(vb),
        _ptr(soft_k, dt, "soft_k"), _ptr(soft_v, dt, "soft_v"),
        _ptr(seq_len, torch.int32, "seq_len"), _ptr(vis, torch.int32, "vis"),
        _ptr(row_flags, torch.uint8, "row_flags"), _ptr(o), _ptr(lse, torch.float32, "lse"),
        _stream(stream)))


def spec_vocab_reduce(logits, proposal, argmax, lse, zprop, stream=None):
    lib = load_library()
    n, V = logits.shape
    _check("spec_vocab_reduce", lib.spec_vocab_reduce(
        _ptr(logits, name="logits"), spec_dtype(logits), n, V,
        _ptr(proposal, torch.int32, "proposal"), _ptr(argmax, torch.int32, "argmax"),
        _ptr(lse, torch.float32, "lse"), _ptr(zprop, torch.float32, "zprop"),
        _stream(stream)))


def spec_accept(desc: AcceptDesc, logits, tokens, tree_parent, row_of, n_nodes, argmax, lse,
                zprop, acc_len, path, next_token, last_node, stream=None):
    lib = load_library()
    i32 = torch.int32
    _check("spec_accept", lib.spec_accept(
        ctypes.byref(desc), _ptr(logits, name="logits"), _ptr(tokens, i32, "tokens"),
        _ptr(tree_parent, i32, "tree_parent"), _ptr(row_of, i32, "row_of"),
        _ptr(n_nodes, i32, "n_nodes"), _ptr(argmax, i32, "argmax"),
        _ptr(lse, torch.float32, "lse"), _ptr(zprop, torch.float32, "zprop"),
        _ptr(acc_len, i32, "acc_len"), _ptr(path, i32, "path"),
        _ptr(next_token, i32, "next_token"), _ptr(last_node, i32, "last_node"),
        _stream(stream)))


def kv_commit(cache: KvDesc, kb, vb, path, acc_len, seq_len, free_pages=None, free_head=None,
              stream=None):
    lib = load_library()
    B, Hkv, R, d = kb.shape
    i32 = torch.int32
    n_free = 0 if free_pages is None else free_pages.numel()
    _check("kv_commit", lib.kv_commit(
        ctypes.byref(cache), B, R, _ptr(kb, name="kb"), _ptr(vb, kb.dtype, "vb"),
        path.shape[1], _ptr(path, i32, "path"), _ptr(acc_len, i32, "acc_len"),
        _ptr(seq_len, i32, "seq_len"), _ptr(free_pages, i32, "free_pages"), n_free,
        _ptr(free_head, i32, "free_head"), _stream(stream)))


def spec_get_status(stream=None) -> int:
    """Synchronise, read and clear the device status word (SPEC_DEV_* bits)."""
    lib = load_library()
    out = ctypes.c_int32(0)
    code = lib.spec_get_status(_stream(stream), ctypes.byref(out))
    if code not in (SPEC_OK, SPEC_ERR_DEVICE):
        _check("spec_get_status", code)
    return out.value


def spec_set_wait_limit(cycles: int) -> int:
    """Limit (SM cycles) of the kernels' pipeline waits from now on; a
    negative value restores the default.  Returns the previous limit."""
    return load_library().spec_set_wait_limit(int(cycles))


def spec_la_prefill_attn(desc: PrefillDesc, q, k, v, o, lse, stream=None):
    """Prefill-form Lookahead Attention: q, o [B][n+k][Hq][d]; k, v
    [B][n+k][Hkv][d] (bf16); lse [B][Hq][n+k] fp32."""
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _ptr(t, torch.bfloat16, name)
    _check("spec_la_prefill_attn", lib.spec_la_prefill_attn(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
        _ptr(lse, torch.float32, "lse"), _stream(stream)))


def spec_accept_soft(desc: SoftDesc, logits, draft_logits, tokens, tree_parent, row_of,
                     child_draft_row, n_nodes, u_accept, u_sample, lse_t, lse_d, acc_len, path,
                     next_token, last_node, stream=None):
    """Soft-matching acceptance (ratio test down the tree, residual draw)."""
    lib = load_library()
    i32, f32 = torch.int32, torch.float32
    _check("spec_accept_soft", lib.spec_accept_soft(
        ctypes.byref(desc), _ptr(logits, name="logits"),
        _ptr(draft_logits, logits.dtype, "draft_logits"), _ptr(tokens, i32, "tokens"),
        _ptr(tree_parent, i32, "tree_parent"), _ptr(row_of, i32, "row_of"),
        _ptr(child_draft_row, i32, "child_draft_row"), _ptr(n_nodes, i32, "n_nodes"),
        _ptr(u_accept, f32, "u_accept"), _ptr(u_sample, f32, "u_sample"),
        _ptr(lse_t, f32, "lse_t"), _ptr(lse_d, f32, "lse_d"), _ptr(acc_len, i32, "acc_len"),
        _ptr(path, i32, "path"), _ptr(next_token, i32, "next_token"),
        _ptr(last_node, i32, "last_node"), _stream(stream)))


def spec_draft_tree(desc: DraftDesc, stream_logits, stream_row, root_token, tokens, tree_parent,
                    n_nodes, vparent=None, stream=None):
    """Top-k per stream -> complete k-ary draft tree (+ the block's vparent)."""
    lib = load_library()
    i32 = torch.int32
    _check("spec_draft_tree", lib.spec_draft_tree(
        ctypes.byref(desc), _ptr(stream_logits, name="stream_logits"),
        _ptr(stream_row, i32, "stream_row"), _ptr(root_token, i32, "root_token"),
        _ptr(tokens, i32, "tokens"), _ptr(tree_parent, i32, "tree_parent"),
        _ptr(n_nodes, i32, "n_nodes"), _ptr(vparent, i32, "vparent"), _stream(stream)))


def spec_prune_tree(desc: PruneDesc, tokens, tree_parent, n_nodes, early_logits, keep_map,
                    tokens_out, parent_out, n_out, vparent=None, stream=None):
    """Drop subtrees whose edge probability under the early-exit logits is
    below the threshold; compact the survivors."""
    lib = load_library()
    i32 = torch.int32
    _check("spec_prune_tree", lib.spec_prune_tree(
        ctypes.byref(desc), _ptr(tokens, i32, "tokens"), _ptr(tree_parent, i32, "tree_parent"),
        _ptr(n_nodes, i32, "n_nodes"), _ptr(early_logits, name="early_logits"),
        _ptr(keep_map, i32, "keep_map"), _ptr(tokens_out, i32, "tokens_out"),
        _ptr(parent_out, i32, "parent_out"), _ptr(n_out, i32, "n_out"),
        _ptr(vparent, i32, "vparent"), _stream(stream)))


def spec_stream_rotate_values(desc: RotateDesc, n_nodes, vb, stream=None):
    """Stream rows of the block values := their node's values rotated by
    e^{i eps s} (in place)."""
    lib = load_library()
    _check("spec_stream_rotate_values", lib.spec_stream_rotate_values(
        ctypes.byref(desc), _ptr(n_nodes, torch.int32, "n_nodes"), _ptr(vb, name="vb"),
        _stream(stream)))


def spec_future_gather(o, last_node, row_offset, out, stream=None):
    """out[b] = o[b][row_offset + last_node[b]] (o: [B][R][...])."""
    lib = load_library()
    B, R = o.shape[0], o.shape[1]
    row = o[0, 0].numel()
    _ptr(out, o.dtype, "out")
    _check("spec_future_gather", lib.spec_future_gather(
        B, R, row, spec_dtype(o), _ptr(o, name="o"), _ptr(last_node, torch.int32, "last_node"),
        row_offset, _ptr(out), _stream(stream)))


# ------------------------------------------------ 8-bit cache, plans, logits

def _on(t, dtype, shape, name, dev, optional=False):
    """Device pointer of a contiguous tensor of this type and shape (None: any)
    on device `dev`, the current one, where the library launches."""
    try:
        if (t.get_device() == dev and (dtype is None or t.dtype is dtype) and
                (shape is None or t.shape == shape) and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:          # not a tensor
        pass
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _cur(stream):
    """Handle of a torch stream (None: the current one), which must belong to
    the current device, and that device's index."""
    # (the bare queries: torch.cuda's own take several times as long, and a
    # Stream object ten times)
    dev = torch._C._cuda_getDevice()
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev), dev
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the current device is cuda:{dev}")
    return stream.cuda_stream, dev


def kv8_desc(kv: torch.Tensor, scales: torch.Tensor, page_table: torch.Tensor = None) -> Kv8Desc:
    """kv: float8_e4m3fn (or uint8) [n_pages][Hkv][page_size / 8][2][8][d];
    scales fp32 [n_pages][Hkv][2]; page_table int32 [B][max_pages] (None for
    kv8_append alone).  The descriptor keeps the tensors alive."""
    if kv.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"kv must be float8_e4m3fn or uint8, got {kv.dtype}")
    if kv.dim() != 6 or kv.shape[3] != 2 or kv.shape[4] != 8:
        raise ValueError("kv must be [n_pages][Hkv][page_size / 8][2][8][d]")
    P, Hkv, groups, _, _, d = kv.shape
    if not kv.is_cuda:
        raise TypeError("kv must be a CUDA tensor")
    dev = kv.get_device()
    _on(kv, None, None, "kv", dev)
    _on(scales, torch.float32, (P, Hkv, 2), "scales", dev)
    B = maxp = 0
    pt = _on(page_table, torch.int32, None, "page_table", dev, optional=True)
    if page_table is not None:
        B, maxp = page_table.shape
    desc = Kv8Desc(Hkv, d, kv.data_ptr(), scales.data_ptr(), B, P, groups * 8, maxp, pt)
    desc.device = dev
    desc.tensors = (kv, scales, page_table)     # (alive as long as the descriptor)
    return desc


def _cache_on(cache, dev):
    if getattr(cache, "device", dev) != dev:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")


def spec_verify_attn_kv8_workspace_size(attn: AttnDesc, cache: Kv8Desc) -> int:
    n = c_size_t(0)
    _check("spec_verify_attn_kv8_workspace_size",
           load_library().spec_verify_attn_kv8_workspace_size(
               ctypes.byref(attn), ctypes.byref(cache), ctypes.byref(n)))
    return n.value


def spec_verify_attn_kv8(attn: AttnDesc, q, cache: Kv8Desc, kb, vb, soft_k, soft_v, seq_len, vis,
                         row_flags, o, lse, workspace, stream=None):
    """spec_verify_attn over a prefix held in 8 bits."""
    st, dev = _cur(stream)
    B, R, Hq, Hkv, d, ns = (attn.batch, attn.n_rows, attn.n_q_heads, attn.n_kv_heads, attn.head_dim,
                            attn.n_soft)
    dt = torch.bfloat16 if attn.dtype == SPEC_BF16 else torch.float32
    _cache_on(cache, dev)
    soft = (Hkv, ns, d)
    if ns == 0:
        soft_k = soft_v = None
    _check("spec_verify_attn_kv8", load_library().spec_verify_attn_kv8(
        ctypes.byref(attn), _on(q, dt, (B, R, Hq, d), "q", dev), ctypes.byref(cache),
        _on(kb, dt, (B, Hkv, R, d), "kb", dev), _on(vb, dt, (B, Hkv, R, d), "vb", dev),
        _on(soft_k, dt, soft, "soft_k", dev, ns == 0), _on(soft_v, dt, soft, "soft_v", dev, ns == 0),
        _on(seq_len, torch.int32, (B,), "seq_len", dev),
        _on(vis, torch.int32, (B, R, (R + 31) // 32), "vis", dev),
        _on(row_flags, torch.uint8, (B, R), "row_flags", dev),
        _on(o, dt, (B, R, Hq, d), "o", dev), _on(lse, torch.float32, (B, Hq, R), "lse", dev),
        _on(workspace, None, None, "workspace", dev), workspace.numel() * workspace.element_size(),
        st))


def kv8_commit(cache: Kv8Desc, kb, vb, path, acc_len, seq_len, free_pages, free_head, stream=None):
    """kv_commit into a cache held in 8 bits."""
    st, dev = _cur(stream)
    _cache_on(cache, dev)
    B, Hkv, R, d = kb.shape
    if (Hkv, d) != (cache.n_kv_heads, cache.head_dim):
        raise ValueError(f"kb must be [B][{cache.n_kv_heads}][R][{cache.head_dim}]")
    i32 = torch.int32
    cap = path.shape[1]
    _check("kv8_commit", load_library().kv8_commit(
        ctypes.byref(cache), spec_dtype(kb), B, R, _on(kb, None, None, "kb", dev),
        _on(vb, kb.dtype, kb.shape, "vb", dev), cap, _on(path, i32, (B, cap), "path", dev),
        _on(acc_len, i32, (B,), "acc_len", dev), _on(seq_len, i32, (B,), "seq_len", dev),
        _on(free_pages, i32, None, "free_pages", dev), free_pages.numel(),
        _on(free_head, i32, (1,), "free_head", dev), st))


def _packed_rows(t, cache, n, name, dev):
    """Pointer and row stride of [n][Hkv][d] rows that may lie in wider rows."""
    return _rows(t, n, cache.n_kv_heads, cache.head_dim, name, dev)


def _rows(t, n, H, d, name, dev, dtype=None):
    """Pointer and row stride of [n][H][d] rows that may lie in wider rows."""
    try:
        if t.get_device() == dev and t.shape == (n, H, d) and (dtype is None or t.dtype is dtype):
            s = t.stride()
            if s[2] == 1 and (H == 1 or s[1] == d):
                return t.data_ptr(), s[0] if n > 1 else H * d
    except AttributeError:          # not a tensor
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    if t.shape != (n, H, d):
        raise ValueError(f"{name} must be {[n, H, d]}, got {list(t.shape)}")
    if n and (t.stride(2) != 1 or (H > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr(), t.stride(0) if n > 1 else H * d


def kv8_append(cache: Kv8Desc, k, v, slot_map, stream=None):
    """Packed new tokens k, v [n][Hkv][d] (rows may be part of wider ones) into
    the slots of slot_map int64 [n] (negative: not written, which the token at
    offset 0 of a new page has to be)."""
    st, dev = _cur(stream)
    _cache_on(cache, dev)
    n = slot_map.numel()
    pk, sk = _packed_rows(k, cache, n, "k", dev)
    pv, sv = _packed_rows(v, cache, n, "v", dev)
    if v.dtype != k.dtype:
        raise TypeError(f"v must be {k.dtype}, got {v.dtype}")
    _check("kv8_append", load_library().kv8_append(
        ctypes.byref(cache), spec_dtype(k), n, pk, sk, pv, sv,
        _on(slot_map, torch.int64, (n,), "slot_map", dev), st))


def spec_page_plan(page_size, n_pages, seq_len, n_new, page_table, free_pages, free_head, cu_new,
                   slot_map, new_len=None, stream=None):
    """Block tables and slot maps for n_new[b] more tokens of each request."""
    st, dev = _cur(stream)
    B, maxp = page_table.shape
    i32 = torch.int32
    _check("spec_page_plan", load_library().spec_page_plan(
        B, page_size, n_pages, maxp, _on(seq_len, i32, (B,), "seq_len", dev),
        _on(n_new, i32, (B,), "n_new", dev), _on(page_table, i32, None, "page_table", dev),
        _on(free_pages, i32, None, "free_pages", dev), free_pages.numel(),
        _on(free_head, i32, (1,), "free_head", dev), _on(cu_new, i32, (B + 1,), "cu_new", dev),
        slot_map.numel(), _on(slot_map, torch.int64, None, "slot_map", dev),
        _on(new_len, i32, (B,), "new_len", dev, True), st))


def logits_desc(batch, n_judge_rows, vocab, logit_dtype, max_nodes=0, hist_cap=0, n_bias=0,
                n_masks=0) -> LogitsDesc:
    return LogitsDesc(batch, n_judge_rows, vocab, logit_dtype, max_nodes, hist_cap, n_bias, n_masks)


def spec_logits_adjust(desc: LogitsDesc, logits, out, history=None, hist_len=None, n_prompt=None,
                       tokens=None, tree_parent=None, row_node=None, repetition=None,
                       presence=None, frequency=None, bias_ids=None, bias=None, mask_bits=None,
                       row_mask=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on judged rows;
    what the descriptor gives no room (0) is not passed."""
    st, dev = _cur(stream)
    B, Rj, V, N, H, nb, nm = (desc.batch, desc.n_judge_rows, desc.vocab, desc.max_nodes,
                              desc.hist_cap, desc.n_bias, desc.n_masks)
    dt = torch.bfloat16 if desc.logit_dtype == SPEC_BF16 else torch.float32
    i32, f32 = torch.int32, torch.float32
    if H == 0:
        history = hist_len = n_prompt = None
    if N == 0:
        tokens = tree_parent = row_node = None
    if nb == 0:
        bias_ids = bias = None
    if nm == 0:
        mask_bits = row_mask = None
    _check("spec_logits_adjust", load_library().spec_logits_adjust(
        ctypes.byref(desc), _on(logits, dt, (B, Rj, V), "logits", dev),
        _on(out, dt, (B, Rj, V), "out", dev), _on(history, i32, (B, H), "history", dev, H == 0),
        _on(hist_len, i32, (B,), "hist_len", dev, H == 0),
        _on(n_prompt, i32, (B,), "n_prompt", dev, True),
        _on(tokens, i32, (B, N), "tokens", dev, N == 0),
        _on(tree_parent, i32, (B, N), "tree_parent", dev, N == 0),
        _on(row_node, i32, (B, Rj), "row_node", dev, True),
        _on(repetition, f32, (B,), "repetition", dev, True),
        _on(presence, f32, (B,), "presence", dev, True),
        _on(frequency, f32, (B,), "frequency", dev, True),
        _on(bias_ids, i32, (B, nb), "bias_ids", dev, nb == 0),
        _on(bias, f32, (B, nb), "bias", dev, nb == 0),
        _on(mask_bits, i32, (nm, (V + 31) // 32), "mask_bits", dev, nm == 0),
        _on(row_mask, i32, (B, Rj), "row_mask", dev, nm == 0), st))


# ------------------------------------- a prompt's chunk: positions, cache, attention

def rope_desc(n_tokens, n_q_heads, n_k_heads, head_dim, rot_dim, layout, dtype,
              attention=1.0) -> RopeDesc:
    return RopeDesc(n_tokens, n_q_heads, n_k_heads, head_dim, rot_dim, layout, dtype, attention)


def spec_rope_freqs(rot_dim, base=10000.0, scaling=SPEC_ROPE_PLAIN, factor=1.0, trained_len=0.0,
                    low=0.0, high=0.0):
    """Rotary frequencies (radians a position) for spec_rope: a ctypes array of
    rot_dim / 2 doubles, on the host."""
    freqs = (c_double * max(1, rot_dim // 2))()
    _check("spec_rope_freqs", load_library().spec_rope_freqs(
        rot_dim, base, scaling, factor, trained_len, low, high, freqs))
    return freqs


def spec_rope(desc: RopeDesc, freqs, q, q_out, k=None, k_out=None, positions=None, seq_len=None,
              cu_new=None, stream=None):
    """Rotary positions of q [n][Hq][d] and k [n][Hk][d] (rows may be part of
    wider ones) into q_out and k_out, which may be q and k themselves.  Positions
    are given (int32 [n], negative: row left as it is), or follow from seq_len
    int32 [B] and cu_new int32 [B + 1].  freqs: from spec_rope_freqs, or any
    sequence of rot_dim / 2 numbers."""
    st, dev = _cur(stream)
    n, Hq, Hk, d = desc.n_tokens, desc.n_q_heads, desc.n_k_heads, desc.head_dim
    half = max(1, desc.rot_dim // 2)
    if len(freqs) != half:
        raise ValueError(f"freqs must have {half} entries, got {len(freqs)}")
    if not isinstance(freqs, ctypes.Array) or freqs._type_ is not c_double:
        freqs = (c_double * half)(*(float(f) for f in freqs))
    dt = torch.bfloat16 if desc.dtype == SPEC_BF16 else torch.float32
    none = (None, 0)
    pq, sq = _rows(q, n, Hq, d, "q", dev, dt) if Hq else none
    pqo, sqo = _rows(q_out, n, Hq, d, "q_out", dev, dt) if Hq else none
    pk, sk = _rows(k, n, Hk, d, "k", dev, dt) if Hk else none
    pko, sko = _rows(k_out, n, Hk, d, "k_out", dev, dt) if Hk else none
    i32, B = torch.int32, 0
    if positions is not None:
        pos, sl, cu = _on(positions, i32, (n,), "positions", dev), None, None
    else:
        sl = _on(seq_len, i32, None, "seq_len", dev)
        B, pos = seq_len.numel(), None
        cu = _on(cu_new, i32, (B + 1,), "cu_new", dev)
    _check("spec_rope", load_library().spec_rope(ctypes.byref(desc), freqs, pq, sq, pqo, sqo, pk, sk, pko, sko,
                                                 pos, B, sl, cu, st))


def kv_append(cache: KvDesc, k, v, slot_map, stream=None):
    """Packed new tokens k, v [n][Hkv][d] (rows may be part of wider ones) into
    the slots of slot_map int64 [n] (negative: not written) of a cache of rows."""
    st, dev = _cur(stream)
    _cache_on(cache, dev)
    n = slot_map.numel()
    pk, sk = _packed_rows(k, cache, n, "k", dev)
    pv, sv = _packed_rows(v, cache, n, "v", dev)
    for name, t in (("k", k), ("v", v)):
        if spec_dtype(t) != cache.dtype:
            raise TypeError(f"{name} must have the cache's dtype, got {t.dtype}")
    _check("kv_append", load_library().kv_append(
        ctypes.byref(cache), n, pk, sk, pv, sv, _on(slot_map, torch.int64, (n,), "slot_map", dev), st))


def chunk_desc(batch, n_tokens, n_q_heads, n_kv_heads, head_dim, dtype, scale=0.0) -> ChunkDesc:
    return ChunkDesc(batch, n_tokens, n_q_heads, n_kv_heads, head_dim, dtype, scale)


def _chunk_size(fn, desc, cache):
    n = c_size_t(0)
    _check(fn, getattr(load_library(), fn)(ctypes.byref(desc), ctypes.byref(cache), ctypes.byref(n)))
    return n.value


def _chunk(fn, desc, q, cache, seq_len, cu_new, o, lse, workspace, stream):
    st, dev = _cur(stream)
    _cache_on(cache, dev)
    B, n, Hq, d = desc.batch, desc.n_tokens, desc.n_q_heads, desc.head_dim
    dt = torch.bfloat16 if desc.dtype == SPEC_BF16 else torch.float32
    pq, sq = _rows(q, n, Hq, d, "q", dev, dt)
    _check(fn, getattr(load_library(), fn)(
        ctypes.byref(desc), pq, sq, ctypes.byref(cache), _on(seq_len, torch.int32, (B,), "seq_len", dev),
        _on(cu_new, torch.int32, (B + 1,), "cu_new", dev), _on(o, dt, (n, Hq, d), "o", dev),
        _on(lse, torch.float32, (n, Hq), "lse", dev), _on(workspace, None, None, "workspace", dev),
        workspace.numel() * workspace.element_size(), st))


def spec_chunk_attn_workspace_size(desc: ChunkDesc, cache: KvDesc) -> int:
    return _chunk_size("spec_chunk_attn_workspace_size", desc, cache)


def spec_chunk_attn(desc: ChunkDesc, q, cache: KvDesc, seq_len, cu_new, o, lse, workspace, stream=None):
    """Attention of packed new tokens q [n][Hq][d] (rows may be part of wider
    ones), which the cache of rows already holds, each over its request's tokens
    up to itself; o [n][Hq][d], lse [n][Hq]."""
    _chunk("spec_chunk_attn", desc, q, cache, seq_len, cu_new, o, lse, workspace, stream)


def spec_chunk_attn_kv8_workspace_size(desc: ChunkDesc, cache: Kv8Desc) -> int:
    return _chunk_size("spec_chunk_attn_kv8_workspace_size", desc, cache)


def spec_chunk_attn_kv8(desc: ChunkDesc, q, cache: Kv8Desc, seq_len, cu_new, o, lse, workspace,
                        stream=None):
    """spec_chunk_attn over a cache held in 8 bits."""
    _chunk("spec_chunk_attn_kv8", desc, q, cache, seq_len, cu_new, o, lse, workspace, stream)
