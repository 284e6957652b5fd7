"""Thin Python binding of libspecdec.so: one function per C-ABI entry point,
with the same names.  Argument marshalling only -- every step runs in the CUDA
kernels behind the C ABI.  Tensors are torch CUDA tensors (torch provides the
device memory and the stream); the current torch stream is used unless a
stream is given.

Importing this module loads the library and raises ``RuntimeError`` if it is
missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libspecdec.so")

SPEC_OK = 0
SPEC_F32, SPEC_BF16 = 0, 1
(OP_SELECT_TOPK, OP_BUILD_TREE, OP_VERIFY_ATTENTION, OP_VERIFY_GREEDY, OP_VERIFY_SAMPLING, OP_COMMIT_KV,
 OP_VERIFY_TARGET_ONLY, OP_ALLOC_SLOTS, OP_COMMIT_KV_Q8, OP_VERIFY_ATTENTION_Q8, OP_TOKEN_LOGPROBS) = range(11)
DEV_INDEX, DEV_INVARIANT, DEV_LENGTH, DEV_TIMEOUT, DEV_SPACE = 1, 2, 4, 8, 16
Q8_EXP_MIN = 16  # smallest scale exponent byte the library writes (the scale is 2^(e - 127))
_ERRORS = {-1: "bad argument", -2: "workspace too small or misaligned", -3: "CUDA launch failed",
           -4: "unsupported dtype or head size"}

EXPORTS = ["spec_workspace_size", "spec_workspace_init", "spec_workspace_set_overlap", "spec_last_error",
           "spec_device_sm_count", "spec_select_topk", "spec_build_tree", "spec_verify_attention",
           "spec_verify_greedy", "spec_verify_sampling", "spec_verify_target_only", "spec_build_chain_tree",
           "spec_verify_chain_greedy", "spec_assign_draft_locs", "spec_duplicate_prefix_tail",
           "spec_build_full_mask", "spec_add_penalties", "spec_renorm_probs", "spec_verify_sampling_probs",
           "spec_verify_target_only_probs", "spec_commit_kv", "spec_alloc_slots", "spec_commit_kv_q8",
           "spec_verify_attention_q8", "spec_token_logprobs", "spec_verify_greedy_noalloc",
           "spec_noalloc_last_error"]


class SpecError(RuntimeError):
    pass


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libspecdec.so is not built ({LIB_PATH}); run `python -m accept_select_top_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
    sig = {
        "spec_workspace_size": (Z, [I, I, I, I, I, I, I, I]),
        "spec_workspace_init": (I, [P, Z, P]),
        "spec_workspace_set_overlap": (I, [P, I]),
        "spec_last_error": (I, [P, P]),
        "spec_device_sm_count": (I, []),
        "spec_select_topk": (I, [I, I, I, I, I, P, F, P, P, P, I, P, I, P, P, P, P, Z, P]),
        "spec_build_tree": (I, [I, I, I, I, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_verify_attention": (I, [I, I, I, I, I, I, P, P, P, L, P, I, I, P, P, I, P, P, F, P, P, P, Z, P]),
        "spec_verify_greedy": (I, [I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_verify_sampling": (I, [I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_verify_target_only": (I, [I, I, I, I, I, P, P, P, P, F, F, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_build_chain_tree": (I, [I, I, P, P, I, P, P, P, P, P, P, P, P]),
        "spec_verify_chain_greedy": (I, [I, I, I, I, P, P, I, P, P, P, P, P, P, P, P, Z, P]),
        "spec_assign_draft_locs": (I, [I, I, I, I, P, I, I, P, P, L, P, P, P, Z, P]),
        "spec_duplicate_prefix_tail": (I, [I, I, I, I, I, I, I, P, P, L, P, I, I, P, P, P, Z, P]),
        "spec_build_full_mask": (I, [I, I, P, P, I, P, Z, P, Z, P]),
        "spec_add_penalties": (I, [I, I, I, I, P, P, P]),
        "spec_renorm_probs": (I, [I, I, I, I, P, P, P, P, P, P]),
        "spec_verify_sampling_probs": (I, [I, I, I, I, P, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_verify_target_only_probs": (I, [I, I, I, I, P, P, P, F, F, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_commit_kv": (I, [I, I, I, I, I, I, I, P, P, L, P, I, I, P, P, P, P, P, P, P, P, P, Z, P]),
        "spec_alloc_slots": (I, [I, I, P, P, P, I, P, I, P, L, P, I, I, P, I, P, P, P, I, P, P, Z, P]),
        "spec_commit_kv_q8": (I, [I, I, I, I, I, P, P, L, L, P, P, P, P, L, P, I, I, P, P, P, P, P, I, P, P, Z, P]),
        "spec_verify_attention_q8": (I, [I, I, I, I, I, I, P, L, P, P, L, P, P, P, P, L, P, I, I, P, P, I, P, F, P, P,
                                         P, Z, P]),
        "spec_token_logprobs": (I, [I, I, I, I, I, P, P, P, P, I, P, P, P, P, P, Z, P]),
        "spec_verify_greedy_noalloc": (I, [I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, P]),
        "spec_noalloc_last_error": (I, [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise SpecError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise SpecError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, what: str):
    if rc != SPEC_OK:
        raise SpecError(f"{what}: {_ERRORS.get(rc, rc)}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise SpecError(f"logits must be float32 or bfloat16, got {t.dtype}")


class Workspace:
    """Caller-owned scratch memory for the C ABI (a zero-filled uint8 tensor)."""

    def __init__(self, nbytes: int, device=None, stream=None):
        self.nbytes = max(int(nbytes), 256)
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        # zero-filled through the C ABI, which also forgets any earlier
        # workspace that lived at this address
        self.address, self.device = self.tensor.data_ptr(), self.tensor.get_device()
        _check(LIB.spec_workspace_init(self.ptr, ctypes.c_size_t(self.nbytes), _stream(stream)),
               "spec_workspace_init")

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())

    def set_overlap(self, enable: bool):
        """Allow (or forbid) a select or greedy accept on this workspace to read
        its main input before the kernel ahead of it has finished.  Off by
        default; see spec_workspace_set_overlap for what the caller asserts."""
        _check(LIB.spec_workspace_set_overlap(self.ptr, 1 if enable else 0), "spec_workspace_set_overlap")

    def last_error(self, stream=None) -> int:
        rc = LIB.spec_last_error(self.ptr, _stream(stream))
        if rc < 0:
            _check(rc, "spec_last_error")
        return rc


def spec_workspace_size(op: int, b: int, n: int, k: int, V: int, Hq: int = 0, Hkv: int = 0,
                        max_seq_len: int = 0) -> int:
    return int(LIB.spec_workspace_size(op, b, n, k, V, Hq, Hkv, max_seq_len))


def spec_device_sm_count() -> int:
    return int(LIB.spec_device_sm_count())


def spec_select_topk(step: int, b: int, k: int, draft_logits: torch.Tensor, temperature: float,
                     scores_in: Optional[torch.Tensor], score_blk: torch.Tensor, token_blk: torch.Tensor,
                     score_ld: int, parent_blk: Optional[torch.Tensor], parent_ld: int,
                     scores_out: torch.Tensor, next_input_ids: torch.Tensor,
                     topk_p_out: Optional[torch.Tensor], ws: Workspace, stream=None):
    V = draft_logits.shape[-1]
    _check(LIB.spec_select_topk(step, b, k, V, _dtype_code(draft_logits), _ptr(draft_logits), float(temperature),
                                _ptr(scores_in), _ptr(score_blk), _ptr(token_blk), score_ld, _ptr(parent_blk),
                                parent_ld, _ptr(scores_out), _ptr(next_input_ids), _ptr(topk_p_out), ws.ptr,
                                ws.nbytes, _stream(stream)), "spec_select_topk")


def spec_build_tree(b: int, k: int, S: int, n: int, score_space, token_space, parent_space, bonus, seq_lens,
                    draft_tokens, positions, retrieve_index, next_token, next_sibling, mask_bits,
                    ws: Workspace, stream=None):
    _check(LIB.spec_build_tree(b, k, S, n, _ptr(score_space), _ptr(token_space), _ptr(parent_space), _ptr(bonus),
                               _ptr(seq_lens), _ptr(draft_tokens), _ptr(positions), _ptr(retrieve_index),
                               _ptr(next_token), _ptr(next_sibling), _ptr(mask_bits), ws.ptr, ws.nbytes,
                               _stream(stream)), "spec_build_tree")


def spec_verify_attention(b: int, n: int, Hq: int, Hkv: int, D: int, page_size: int, q, k_pool, v_pool,
                          req_to_token, req_pool_idx, seq_lens, max_seq_len: int, verify_loc, mask_bits,
                          scale: float, out, lse, ws: Workspace, stream=None):
    num_slots = k_pool.shape[0]
    _check(LIB.spec_verify_attention(b, n, Hq, Hkv, D, page_size, _ptr(q), _ptr(k_pool), _ptr(v_pool), num_slots,
                                     _ptr(req_to_token), req_to_token.shape[0], req_to_token.shape[1],
                                     _ptr(req_pool_idx), _ptr(seq_lens), int(max_seq_len), _ptr(verify_loc),
                                     _ptr(mask_bits), float(scale), _ptr(out), _ptr(lse), ws.ptr, ws.nbytes,
                                     _stream(stream)), "spec_verify_attention")


def spec_verify_greedy(b: int, n: int, S: int, logits, draft_tokens, retrieve_index, next_token, next_sibling,
                       predict, accept_index, accept_lens, accepted_tokens, next_root, ws: Workspace, stream=None):
    V = logits.shape[-1]
    _check(LIB.spec_verify_greedy(b, n, S, V, _dtype_code(logits), _ptr(logits), _ptr(draft_tokens),
                                  _ptr(retrieve_index), _ptr(next_token), _ptr(next_sibling), _ptr(predict),
                                  _ptr(accept_index), _ptr(accept_lens), _ptr(accepted_tokens), _ptr(next_root),
                                  ws.ptr, ws.nbytes, _stream(stream)), "spec_verify_greedy")


def spec_verify_sampling(b: int, n: int, S: int, logits, draft_probs, temperatures, u, u_final, draft_tokens,
                         retrieve_index, next_token, next_sibling, predict, accept_index, accept_lens,
                         accepted_tokens, next_root, ws: Workspace, stream=None):
    V = logits.shape[-1]
    _check(LIB.spec_verify_sampling(b, n, S, V, _dtype_code(logits), _ptr(logits), _ptr(draft_probs),
                                    _ptr(temperatures), _ptr(u), _ptr(u_final), _ptr(draft_tokens),
                                    _ptr(retrieve_index), _ptr(next_token), _ptr(next_sibling), _ptr(predict),
                                    _ptr(accept_index), _ptr(accept_lens), _ptr(accepted_tokens), _ptr(next_root),
                                    ws.ptr, ws.nbytes, _stream(stream)), "spec_verify_sampling")


def spec_verify_target_only(b: int, n: int, S: int, logits, temperatures, coins, u_final, threshold_single: float,
                            threshold_acc: float, draft_tokens, retrieve_index, next_token, next_sibling, predict,
                            accept_index, accept_lens, accepted_tokens, next_root, ws: Workspace, stream=None):
    V = logits.shape[-1]
    _check(LIB.spec_verify_target_only(b, n, S, V, _dtype_code(logits), _ptr(logits), _ptr(temperatures),
                                       _ptr(coins), _ptr(u_final), float(threshold_single), float(threshold_acc),
                                       _ptr(draft_tokens), _ptr(retrieve_index), _ptr(next_token),
                                       _ptr(next_sibling), _ptr(predict), _ptr(accept_index), _ptr(accept_lens),
                                       _ptr(accepted_tokens), _ptr(next_root), ws.ptr, ws.nbytes, _stream(stream)),
           "spec_verify_target_only")


def spec_build_chain_tree(b: int, S: int, bonus, draft_tokens, draft_ld: int, seq_lens, tree_tokens, positions,
                          retrieve_index, next_token, next_sibling, mask_bits, stream=None):
    _check(LIB.spec_build_chain_tree(b, S, _ptr(bonus), _ptr(draft_tokens), int(draft_ld), _ptr(seq_lens),
                                     _ptr(tree_tokens), _ptr(positions), _ptr(retrieve_index), _ptr(next_token),
                                     _ptr(next_sibling), _ptr(mask_bits), _stream(stream)), "spec_build_chain_tree")


def spec_verify_chain_greedy(b: int, S: int, logits, draft_tokens, draft_ld: int, prefix_lens, correct_len, bonus,
                             out_tokens, commit_lens, new_seq_lens, accept_index, ws: Workspace, stream=None):
    V = logits.shape[-1]
    _check(LIB.spec_verify_chain_greedy(b, S, V, _dtype_code(logits), _ptr(logits), _ptr(draft_tokens),
                                        int(draft_ld), _ptr(prefix_lens), _ptr(correct_len), _ptr(bonus),
                                        _ptr(out_tokens), _ptr(commit_lens), _ptr(new_seq_lens), _ptr(accept_index),
                                        ws.ptr, ws.nbytes, _stream(stream)), "spec_verify_chain_greedy")


def spec_assign_draft_locs(b: int, topk: int, S: int, page_size: int, req_to_token, req_pool_idx, seq_lens,
                           num_slots: int, out_cache_loc, positions, ws: Workspace, stream=None):
    _check(LIB.spec_assign_draft_locs(b, topk, S, page_size, _ptr(req_to_token), req_to_token.shape[0],
                                      req_to_token.shape[1], _ptr(req_pool_idx), _ptr(seq_lens), int(num_slots),
                                      _ptr(out_cache_loc), _ptr(positions), ws.ptr, ws.nbytes, _stream(stream)),
           "spec_assign_draft_locs")


def spec_duplicate_prefix_tail(b: int, topk: int, S: int, page_size: int, Hkv: int, D: int,
                               k_layers: Sequence[torch.Tensor], v_layers: Sequence[torch.Tensor], req_to_token,
                               req_pool_idx, seq_lens, ws: Workspace, stream=None):
    L = len(k_layers)
    for t in list(k_layers) + list(v_layers):
        _ptr(t)
    kp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_layers])
    vp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_layers])
    _check(LIB.spec_duplicate_prefix_tail(b, topk, S, page_size, Hkv, D, L, ctypes.cast(kp, ctypes.c_void_p),
                                          ctypes.cast(vp, ctypes.c_void_p), k_layers[0].shape[0],
                                          _ptr(req_to_token), req_to_token.shape[0], req_to_token.shape[1],
                                          _ptr(req_pool_idx), _ptr(seq_lens), ws.ptr, ws.nbytes, _stream(stream)),
           "spec_duplicate_prefix_tail")


def spec_build_full_mask(b: int, n: int, seq_lens, mask_bits, fill_prefix: bool, mask, ws: Workspace,
                         stream=None):
    """mask: a uint8 tensor of at least sum_b n*(L_b + n) bytes."""
    _check(LIB.spec_build_full_mask(b, n, _ptr(seq_lens), _ptr(mask_bits), 1 if fill_prefix else 0, _ptr(mask),
                                    ctypes.c_size_t(mask.numel()), ws.ptr, ws.nbytes, _stream(stream)),
           "spec_build_full_mask")


def spec_add_penalties(b: int, n: int, logits, penalties, stream=None):
    """In place: each request's penalty row [b, V] fp32 added to its n verify rows."""
    V = logits.shape[-1]
    _check(LIB.spec_add_penalties(b, n, V, _dtype_code(logits), _ptr(logits), _ptr(penalties), _stream(stream)),
           "spec_add_penalties")


def spec_renorm_probs(b: int, n: int, logits, temperatures, top_k, top_p, probs, stream=None):
    V = logits.shape[-1]
    _check(LIB.spec_renorm_probs(b, n, V, _dtype_code(logits), _ptr(logits), _ptr(temperatures), _ptr(top_k),
                                 _ptr(top_p), _ptr(probs), _stream(stream)), "spec_renorm_probs")


def spec_verify_sampling_probs(b: int, n: int, S: int, probs, draft_probs, u, u_final, draft_tokens, retrieve_index,
                               next_token, next_sibling, predict, accept_index, accept_lens, accepted_tokens,
                               next_root, ws: Workspace, stream=None):
    V = probs.shape[-1]
    _check(LIB.spec_verify_sampling_probs(b, n, S, V, _ptr(probs), _ptr(draft_probs), _ptr(u), _ptr(u_final),
                                          _ptr(draft_tokens), _ptr(retrieve_index), _ptr(next_token),
                                          _ptr(next_sibling), _ptr(predict), _ptr(accept_index), _ptr(accept_lens),
                                          _ptr(accepted_tokens), _ptr(next_root), ws.ptr, ws.nbytes,
                                          _stream(stream)), "spec_verify_sampling_probs")


def spec_verify_target_only_probs(b: int, n: int, S: int, probs, coins, u_final, threshold_single: float,
                                  threshold_acc: float, draft_tokens, retrieve_index, next_token, next_sibling,
                                  predict, accept_index, accept_lens, accepted_tokens, next_root, ws: Workspace,
                                  stream=None):
    V = probs.shape[-1]
    _check(LIB.spec_verify_target_only_probs(b, n, S, V, _ptr(probs), _ptr(coins), _ptr(u_final),
                                             float(threshold_single), float(threshold_acc), _ptr(draft_tokens),
                                             _ptr(retrieve_index), _ptr(next_token), _ptr(next_sibling),
                                             _ptr(predict), _ptr(accept_index), _ptr(accept_lens),
                                             _ptr(accepted_tokens), _ptr(next_root), ws.ptr, ws.nbytes,
                                             _stream(stream)), "spec_verify_target_only_probs")


def spec_commit_kv(b: int, n: int, W: int, Hkv: int, D: int, page_size: int, k_layers: Sequence[torch.Tensor],
                   v_layers: Sequence[torch.Tensor], req_to_token, req_pool_idx, seq_lens, verify_loc,
                   accept_index, accept_lens, new_seq_lens, free_ids, n_free, ws: Workspace, stream=None):
    L = len(k_layers)
    kp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_layers])
    vp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_layers])
    for t in list(k_layers) + list(v_layers):
        _ptr(t)
    _check(LIB.spec_commit_kv(b, n, W, Hkv, D, L, page_size, ctypes.cast(kp, ctypes.c_void_p),
                              ctypes.cast(vp, ctypes.c_void_p), k_layers[0].shape[0], _ptr(req_to_token),
                              req_to_token.shape[0], req_to_token.shape[1], _ptr(req_pool_idx), _ptr(seq_lens),
                              _ptr(verify_loc), _ptr(accept_index), _ptr(accept_lens), _ptr(new_seq_lens),
                              _ptr(free_ids), _ptr(n_free), ws.ptr, ws.nbytes, _stream(stream)), "spec_commit_kv")


# ------------------------------------------------ the 8-bit paged cache, token log probabilities
#
# These calls check what a wrong tensor would turn into a stray access: type,
# device, contiguity and the number of elements the sizes call for.

_I32, _F32, _I64, _BF16 = torch.int32, torch.float32, torch.int64, torch.bfloat16
_E4M3 = torch.float8_e4m3fn


def _in(t: torch.Tensor, dtype, least: int, dev: int, what: str) -> int:
    """Address of a contiguous tensor of `dtype` with at least `least` elements on device `dev`."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= least:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise SpecError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise SpecError(f"{what}: expected a tensor on the current CUDA device")
    if not t.is_contiguous():
        raise SpecError(f"{what}: expected a contiguous tensor")
    raise SpecError(f"{what}: {t.numel()} elements, {least} are needed")


def _pages_in(t: torch.Tensor, shape, dev: int, what: str) -> int:
    """Address of e4m3 pages [num_pages, Hkv, page_size, D] (float8_e4m3fn, or their bytes)."""
    if t.dim() != 4 or t.shape[1:] != shape:
        raise SpecError(f"{what}: expected [num_pages, {', '.join(map(str, shape))}], got {tuple(t.shape)}")
    return _bytes_in(t, dev, what)


def _bytes_in(t: torch.Tensor, dev: int, what: str) -> int:
    """Address of e4m3 values (or their bytes) of a shape that is known to be right."""
    if t.dtype is not _E4M3 and t.dtype is not torch.uint8:
        raise SpecError(f"{what}: expected float8_e4m3fn or uint8, got {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous():
        raise SpecError(f"{what}: expected a contiguous tensor on the current CUDA device")
    return t.data_ptr()


def _rows_in(t: torch.Tensor, heads: int, D: int, least: int, dev: int, what: str):
    """Address and row stride of bf16 rows [rows, heads, D]; the rows may be a view of wider ones."""
    if t.dtype is not _BF16:
        raise SpecError(f"{what}: expected {_BF16}, got {t.dtype}")
    rows, h, d = t.shape
    if h != heads or d != D or rows < least:
        raise SpecError(f"{what}: expected at least {least} rows [{heads}, {D}], got {tuple(t.shape)}")
    ld, sh, sd = t.stride()
    if (sd != 1 and d > 1) or (sh != D and h > 1) or (rows > 1 and ld < heads * D):
        raise SpecError(f"{what}: expected each row's [{heads}, {D}] contiguous")
    if t.get_device() != dev:
        raise SpecError(f"{what}: expected a tensor on the current CUDA device")
    return t.data_ptr(), (ld if rows > 1 else heads * D)


def _workspace_in(ws: Workspace, dev: int) -> int:
    """Address of a workspace on device `dev`."""
    if ws.device != dev:
        raise SpecError(f"workspace: on device {ws.device}, the current CUDA device is {dev}")
    return ws.address


def _device() -> int:
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else torch.cuda.current_device()


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


class LayerList:
    """One tensor a layer, all of one shape, type and strides, with the host array of their
    addresses that the calls over every layer take (built once; the tensors are kept alive)."""

    def __init__(self, tensors: Sequence[torch.Tensor]):
        self.tensors = list(tensors)
        if not self.tensors:
            raise SpecError("a layer list needs at least one layer")
        t0 = self.tensors[0]
        for t in self.tensors[1:]:
            if t.shape != t0.shape or t.dtype != t0.dtype or t.stride() != t0.stride() or t.device != t0.device:
                raise SpecError("the layers of a list must have one shape, type, stride and device")
        self.first = t0
        self.array = (ctypes.c_void_p * len(self.tensors))(*[t.data_ptr() for t in self.tensors])
        self.ptr = ctypes.addressof(self.array)
        self.rows = t0.shape[0] if t0.dim() else 0
        self._checked = {}

    def check(self, fn, *args):
        """fn(first layer, *args), once for each args: addresses and layouts are those of the list's making."""
        got = self._checked.get(args)
        if got is None:
            got = self._checked[args] = fn(self.first, *args)
        return got

    def __len__(self):
        return len(self.tensors)


def _layers(x) -> LayerList:
    return x if isinstance(x, LayerList) else LayerList(x)


def spec_alloc_slots(b: int, page_size: int, req_pool_idx, seq_lens, new_lens, max_new: int, free_ids, n_free,
                     num_slots: int, page_table, req_to_token, cu_new, slot_map, positions, n_left, ws: Workspace,
                     stream=None):
    """Pages for new_lens[b] more tokens a request from the free list (a stack: n_free[0] ids); see
    the header.  num_slots is the pool's size in tokens; req_to_token may be None; n_left may be n_free."""
    dev = _device()
    slots = min(slot_map.numel(), positions.numel())
    width = 0
    if req_to_token is not None:
        width = req_to_token.shape[1]
        if req_to_token.shape[0] != page_table.shape[0]:
            raise SpecError("req_to_token and page_table must have the same rows")
    rows, row_pages = page_table.shape
    _check(LIB.spec_alloc_slots(
        b, page_size, _in(req_pool_idx, _I32, b, dev, "req_pool_idx"), _in(seq_lens, _I32, b, dev, "seq_lens"),
        _in(new_lens, _I32, b, dev, "new_lens"), max_new, _in(free_ids, _I32, 0, dev, "free_ids"), free_ids.numel(),
        _in(n_free, _I32, 1, dev, "n_free"), num_slots // page_size if page_size > 0 else 0,
        _in(page_table, _I32, 1, dev, "page_table"), rows, row_pages,
        None if req_to_token is None else _in(req_to_token, _I32, 1, dev, "req_to_token"), width,
        _in(cu_new, _I32, b + 1, dev, "cu_new"), _in(slot_map, _I32, 0, dev, "slot_map"),
        _in(positions, _I32, 0, dev, "positions"), slots, _in(n_left, _I32, 1, dev, "n_left"),
        _workspace_in(ws, dev), ws.nbytes, _raw_stream(stream, dev)), "spec_alloc_slots")


def spec_commit_kv_q8(b: int, Hkv: int, D: int, page_size: int, k_new, v_new, k_pages, v_pages, k_scales, v_scales,
                      page_table, req_pool_idx, seq_lens, src_index, src_start, lens, max_len: int, new_seq_lens,
                      ws: Workspace, stream=None):
    """Quantises bf16 rows into the e4m3 pages of every layer.  k_new .. v_scales: one tensor a layer
    (a sequence, or a LayerList kept by the caller).  src_index [b, max_len] (accept_index) or
    src_start [b]; the other may be None.  new_seq_lens shares no memory with the arrays of lengths."""
    dev = _device()
    k_new, v_new, k_pages, v_pages = _layers(k_new), _layers(v_new), _layers(k_pages), _layers(v_pages)
    k_scales, v_scales = _layers(k_scales), _layers(v_scales)
    layers = len(k_new)
    if not all(len(x) == layers for x in (v_new, k_pages, v_pages, k_scales, v_scales)):
        raise SpecError("every layer list must have the same length")
    num_rows, num_pages = k_new.rows, k_pages.rows
    _, ld = k_new.check(_rows_in, Hkv, D, 1, dev, "k_new")
    _, ldv = v_new.check(_rows_in, Hkv, D, num_rows, dev, "v_new")
    if ldv != ld:
        raise SpecError("k_new and v_new must have one row stride")
    shape = (Hkv, page_size, D)
    k_pages.check(_pages_in, shape, dev, "k_pages")
    v_pages.check(_pages_in, shape, dev, "v_pages")
    if v_pages.rows != num_pages:
        raise SpecError("k_pages and v_pages must have as many pages")
    k_scales.check(_in, torch.uint8, num_pages * Hkv, dev, "k_scales")
    v_scales.check(_in, torch.uint8, num_pages * Hkv, dev, "v_scales")
    rows, row_pages = page_table.shape
    _check(LIB.spec_commit_kv_q8(
        b, Hkv, D, page_size, layers, k_new.ptr, v_new.ptr, num_rows, ld, k_pages.ptr, v_pages.ptr, k_scales.ptr,
        v_scales.ptr, num_pages, _in(page_table, _I32, 1, dev, "page_table"), rows, row_pages,
        _in(req_pool_idx, _I32, b, dev, "req_pool_idx"), _in(seq_lens, _I32, b, dev, "seq_lens"),
        None if src_index is None else _in(src_index, _I32, b * max_len, dev, "src_index"),
        None if src_start is None else _in(src_start, _I32, b, dev, "src_start"), _in(lens, _I32, b, dev, "lens"),
        max_len, _in(new_seq_lens, _I32, b, dev, "new_seq_lens"), _workspace_in(ws, dev), ws.nbytes,
        _raw_stream(stream, dev)),
        "spec_commit_kv_q8")


def spec_verify_attention_q8(b: int, n: int, Hq: int, Hkv: int, D: int, page_size: int, q, k_new, v_new, k_pages,
                             v_pages, k_scales, v_scales, page_table, req_pool_idx, seq_lens, max_seq_len: int,
                             mask_bits, scale: float, out, lse, ws: Workspace, stream=None):
    """Verify attention over the e4m3 pages and the step's own bf16 rows; q, k_new and v_new
    ([b*n, heads, D]) may be views of one packed projection.  lse may be None."""
    dev = _device()
    rows = b * n
    qp, q_ld = _rows_in(q, Hq, D, rows, dev, "q")
    kp, ld = _rows_in(k_new, Hkv, D, rows, dev, "k_new")
    vp, ldv = _rows_in(v_new, Hkv, D, rows, dev, "v_new")
    if ldv != ld:
        raise SpecError("k_new and v_new must have one row stride")
    pages = k_pages.shape
    if v_pages.shape != pages:
        raise SpecError("k_pages and v_pages must have as many pages")
    num_pages = pages[0] if pages else 0
    shape = (num_pages, Hkv, page_size, D)
    if pages != shape:
        raise SpecError(f"k_pages: expected [num_pages, {Hkv}, {page_size}, {D}], got {tuple(pages)}")
    table_rows, row_pages = page_table.shape
    _check(LIB.spec_verify_attention_q8(
        b, n, Hq, Hkv, D, page_size, qp, q_ld, kp, vp, ld, _bytes_in(k_pages, dev, "k_pages"),
        _bytes_in(v_pages, dev, "v_pages"), _in(k_scales, torch.uint8, num_pages * Hkv, dev, "k_scales"),
        _in(v_scales, torch.uint8, num_pages * Hkv, dev, "v_scales"), num_pages,
        _in(page_table, _I32, 1, dev, "page_table"), table_rows, row_pages,
        _in(req_pool_idx, _I32, b, dev, "req_pool_idx"), _in(seq_lens, _I32, b, dev, "seq_lens"), max_seq_len,
        _in(mask_bits, _I64, rows, dev, "mask_bits"), scale, _in(out, _BF16, rows * Hq * D, dev, "out"),
        None if lse is None else _in(lse, _F32, rows * Hq, dev, "lse"), _workspace_in(ws, dev), ws.nbytes,
        _raw_stream(stream, dev)), "spec_verify_attention_q8")


def spec_token_logprobs(b: int, n: int, W: int, logits, row_index, tokens, temperatures, k: int, logprobs, entropy,
                        top_ids, top_logprobs, ws: Workspace, stream=None):
    """Log probabilities of tokens [b, W] at verify rows row_index [b, W] (accept_index; None: b*n + j),
    entropy (None: not wanted) and the k best alternatives."""
    dev = _device()
    V = logits.shape[-1]
    rows = b * W
    _check(LIB.spec_token_logprobs(
        b, n, W, V, _dtype_code(logits), _in(logits, logits.dtype, b * n * V, dev, "logits"),
        None if row_index is None else _in(row_index, _I32, rows, dev, "row_index"),
        _in(tokens, _I32, rows, dev, "tokens"),
        None if temperatures is None else _in(temperatures, _F32, b, dev, "temperatures"), k,
        _in(logprobs, _F32, rows, dev, "logprobs"),
        None if entropy is None else _in(entropy, _F32, rows, dev, "entropy"),
        None if top_ids is None else _in(top_ids, _I32, rows * k, dev, "top_ids"),
        None if top_logprobs is None else _in(top_logprobs, _F32, rows * k, dev, "top_logprobs"),
        _workspace_in(ws, dev), ws.nbytes, _raw_stream(stream, dev)), "spec_token_logprobs")


def spec_verify_greedy_noalloc(b: int, n: int, S: int, logits, draft_tokens, retrieve_index, next_token,
                               next_sibling, predict, accept_index, accept_lens, accepted_tokens, next_root,
                               stream=None):
    """spec_verify_greedy for callers that cannot allocate device memory: the
    library's fixed device scratch array stands in for the workspace."""
    V = logits.shape[-1]
    _check(LIB.spec_verify_greedy_noalloc(b, n, S, V, _dtype_code(logits), _ptr(logits), _ptr(draft_tokens),
                                          _ptr(retrieve_index), _ptr(next_token), _ptr(next_sibling), _ptr(predict),
                                          _ptr(accept_index), _ptr(accept_lens), _ptr(accepted_tokens),
                                          _ptr(next_root), _stream(stream)), "spec_verify_greedy_noalloc")


def spec_noalloc_last_error(stream=None) -> int:
    """Reads and clears the SPEC_DEV_* bits set by spec_verify_greedy_noalloc
    calls on the current device (synchronises the stream)."""
    rc = LIB.spec_noalloc_last_error(_stream(stream))
    if rc < 0:
        _check(rc, "spec_noalloc_last_error")
    return rc
