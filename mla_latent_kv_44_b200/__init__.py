"""Python binding of libmla (MLA absorbed decode for B200, sm_100a).

Argument marshalling only: every step of the computation runs in the CUDA kernels of
``libmla.so``. Tensors are passed as raw device pointers; PyTorch provides device memory and
streams. The library is loaded on the first call (so that the build step can import this
package before the library exists); that call fails loudly when the library has not been
built (``python -m mla_latent_kv_44_b200.build``). There is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla.so")
# The same library built with a test define that leaves out one K-slab load of the attention
# kernel's first work range (tests of the bounded-wait path load it instead of LIB_PATH).
TEST_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla_testhook.so")

MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA, MLA_ERR_WORKSPACE = range(5)
STATIC_WORKSPACE_BYTES = 40 << 20
MLA_F32, MLA_BF16 = 0, 1
DECODE_AUTO, DECODE_SIMT, DECODE_TENSOR = 0, 1, 2
DEV_OOB_BLOCK, DEV_OOB_POS, DEV_WAIT_TIMEOUT, DEV_BAD_LENGTH = 1, 2, 4, 8
DEV_BAD_TREE, DEV_NO_BLOCKS = 16, 32
STAGE_PLAN, STAGE_ATTEND, STAGE_COMBINE = 1, 2, 4
STAGES_ALL = STAGE_PLAN | STAGE_ATTEND | STAGE_COMBINE
MAX_COMBINE_PARTS = 256  # MLA_MAX_COMBINE_PARTS
MAX_TABLE_BATCH, MAX_TREE = 8192, 256  # MLA_MAX_TABLE_BATCH, MLA_MAX_TREE

_c_i32, _c_f32, _vp, _sz = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t


class MlaConfig(ctypes.Structure):
    _fields_ = [("num_heads", _c_i32), ("head_dim", _c_i32), ("head_dim_v", _c_i32),
                ("kv_rank", _c_i32), ("rope_dim", _c_i32), ("block_size", _c_i32),
                ("rope_base", _c_f32), ("rms_eps", _c_f32), ("softmax_scale", _c_f32),
                ("dtype", _c_i32), ("decode_kernel", _c_i32)]


class MlaFrontConfig(ctypes.Structure):
    _fields_ = [("d_model", _c_i32), ("q_rank", _c_i32), ("q_rms_eps", _c_f32)]


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m mla_latent_kv_44_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(MlaConfig)
    sig = {
        "mla_absorb_query": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "mla_append_latent": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _vp,
                                       _c_i32, _c_i32, _vp, _vp]),
        "mla_decode_workspace_size": (_sz, [P, _c_i32, _c_i32]),
        "mla_decode": (_c_i32, [P, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _c_i32, _c_i32, _vp, _sz,
                                _vp, _vp, _vp, _vp]),
        "mla_decode_stages": (_c_i32, [P, _c_i32, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _c_i32,
                                       _c_i32, _vp, _sz, _vp, _vp, _vp, _vp]),
        "mla_output": (_c_i32, [P, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "mla_decode_static_workspace": (_c_i32, [P, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _c_i32,
                                                 _c_i32, _vp, _vp, _vp, _vp]),
        "mla_decode_step": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _vp,
                                     _c_i32, _vp, _c_i32, _c_i32, _vp, _vp, _sz, _vp, _vp, _vp,
                                     _vp, _vp, _vp]),
        "mla_combine_partials": (_c_i32, [P, _vp, _vp, _c_i32, _c_i32, _vp, _vp, _vp]),
        "mla_append_latent_fp8": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _vp,
                                           _vp, _c_i32, _c_i32, _vp, _vp]),
        "mla_decode_fp8_workspace_size": (_sz, [P, _c_i32, _c_i32, _c_i32]),
        "mla_decode_fp8": (_c_i32, [P, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _c_i32, _c_i32,
                                    _vp, _sz, _vp, _vp, _vp, _vp]),
        "mla_prefill_workspace_size": (_sz, [P, _c_i32]),
        "mla_prefill": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32,
                                 _vp, _vp, _sz, _vp, _vp]),
        "mla_project_workspace_size": (_sz, [P, ctypes.POINTER(MlaFrontConfig), _c_i32]),
        "mla_project": (_c_i32, [P, ctypes.POINTER(MlaFrontConfig), _vp, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _vp, _sz, _vp, _vp]),
        "mla_build_tables": (_c_i32, [P, _vp, _vp, _c_i32, _vp, _c_i32, _vp, _vp, _vp, _c_i32, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _c_i32, _vp, _vp]),
        "mla_tree_masks": (_c_i32, [_vp, _c_i32, _vp, _c_i32, _c_i32, _vp, _vp, _vp, _vp]),
        "mla_append_slots": (_c_i32, [P, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _vp]),
        "mla_decode_tree_workspace_size": (_sz, [P, _c_i32, _c_i32]),
        "mla_decode_tree": (_c_i32, [P, _vp, _vp, _vp, _c_i32, _c_i32, _vp, _c_i32, _c_i32, _vp,
                                     _vp, _vp, _sz, _vp, _vp, _vp, _vp]),
        "mla_commit_tree": (_c_i32, [P, _vp, _vp, _c_i32, _c_i32, _vp, _c_i32, _vp, _c_i32, _vp,
                                     _vp, _c_i32, _vp, _vp]),
        "mla_status_string": (ctypes.c_char_p, [_c_i32]),
        "mla_abi_version": (_c_i32, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


class _Lib:
    """libmla.so, loaded on first use."""

    _handle = None

    def __getattr__(self, name):
        if _Lib._handle is None:
            _Lib._handle = _load()
        fn = getattr(_Lib._handle, name)
        self.__dict__[name] = fn  # found without this call from now on
        return fn


lib = _Lib()


@dataclass
class Config:
    """Shape and numerics of one MLA layer's decode (mirrors ``mla_config``)."""

    num_heads: int
    head_dim: int
    kv_rank: int
    rope_dim: int
    block_size: int
    dtype: str = "bf16"            # "bf16" or "f32"
    head_dim_v: int = 0            # 0: same as head_dim
    rope_base: float = 10000.0
    rms_eps: float = 1e-6
    softmax_scale: float = 0.0     # 0: 1 / sqrt(head_dim + rope_dim)
    decode_kernel: int = DECODE_AUTO

    def c(self) -> MlaConfig:
        scale = self.softmax_scale or 1.0 / math.sqrt(self.head_dim + self.rope_dim)
        return MlaConfig(self.num_heads, self.head_dim, self.head_dim_v or self.head_dim,
                         self.kv_rank, self.rope_dim, self.block_size, self.rope_base,
                         self.rms_eps, scale, MLA_BF16 if self.dtype == "bf16" else MLA_F32,
                         self.decode_kernel)

    def ref(self):
        """A reference to the C struct for a call; built again only when a field has changed."""
        key = (self.num_heads, self.head_dim, self.kv_rank, self.rope_dim, self.block_size,
               self.dtype, self.head_dim_v, self.rope_base, self.rms_eps, self.softmax_scale,
               self.decode_kernel)
        held = self.__dict__.get("_ref")
        if held is None or held[0] != key:
            held = (key, ctypes.byref(self.c()))
            self.__dict__["_ref"] = held
        return held[1]

    @property
    def row_width(self) -> int:
        return self.kv_rank + self.rope_dim

    @property
    def torch_dtype(self):
        import torch
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32


def status_string(status: int) -> str:
    return lib.mla_status_string(status).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(st: int, where: str):
    if st != MLA_OK:
        raise MlaError(st, where)


def absorb_query(cfg: Config, q_nope, q_rope, pos, w_uk, q_out, stream=None, dev_err=None):
    """mla_absorb_query: q_out[n, h] = [W_UK[h]^T q_nope[n, h] || RoPE(q_rope[n, h], pos[n])]."""
    c = cfg.c()
    _check(lib.mla_absorb_query(ctypes.byref(c), _ptr(q_nope), _ptr(q_rope), _ptr(pos),
                                _ptr(w_uk), _ptr(q_out), int(q_nope.shape[0]), _ptr(dev_err),
                                _stream(stream)), "mla_absorb_query")


def append_latent(cfg: Config, ckv_raw, krope_raw, gamma, seq_idx, pos, block_table, pool,
                  dev_err, stream=None):
    """mla_append_latent: write [RMSNorm(c_kv) * gamma || RoPE(k_rope)] rows into the pool."""
    c = cfg.c()
    _check(lib.mla_append_latent(ctypes.byref(c), _ptr(ckv_raw), _ptr(krope_raw), _ptr(gamma),
                                 _ptr(seq_idx), _ptr(pos), _ptr(block_table),
                                 int(block_table.shape[0]), int(block_table.shape[1]), _ptr(pool),
                                 int(pool.shape[0]), int(ckv_raw.shape[0]), _ptr(dev_err),
                                 _stream(stream)), "mla_append_latent")


def decode_workspace_size(cfg: Config, batch: int, q_per_seq: int) -> int:
    c = cfg.c()
    return int(lib.mla_decode_workspace_size(ctypes.byref(c), batch, q_per_seq))


def decode(cfg: Config, q, pool, block_table, seq_lens, q_per_seq: int, workspace, out_latent,
           lse, dev_err, stream=None, stages: int = STAGES_ALL):
    """mla_decode (or a subset of its stages): split-KV absorbed attention over the pool."""
    c = cfg.c()
    _check(lib.mla_decode_stages(ctypes.byref(c), stages, _ptr(q), _ptr(pool), _ptr(block_table),
                                 int(block_table.shape[1]), int(pool.shape[0]), _ptr(seq_lens),
                                 int(seq_lens.shape[0]), q_per_seq, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _ptr(out_latent),
                                 _ptr(lse), _ptr(dev_err), _stream(stream)), "mla_decode")


def decode_static_workspace(cfg: Config, q, pool, block_table, seq_lens, q_per_seq: int,
                            out_latent, lse, dev_err, stream=None):
    """mla_decode_static_workspace: mla_decode with the library's own fixed device workspace,
    for callers that cannot allocate device memory (see include/mla.h)."""
    c = cfg.c()
    _check(lib.mla_decode_static_workspace(ctypes.byref(c), _ptr(q), _ptr(pool),
                                           _ptr(block_table), int(block_table.shape[1]),
                                           int(pool.shape[0]), _ptr(seq_lens),
                                           int(seq_lens.shape[0]), q_per_seq, _ptr(out_latent),
                                           _ptr(lse), _ptr(dev_err), _stream(stream)),
           "mla_decode_static_workspace")


def decode_step(cfg: Config, q_nope, q_rope, w_uk, ckv_raw, krope_raw, gamma, seq_idx, pos,
                block_table, pool, seq_lens, q_per_seq: int, q_work, workspace, out_latent, lse,
                w_uv, o, dev_err, stream=None):
    """mla_decode_step: absorb, append, decode and output of one step in one call (see
    include/mla.h); batch = seq_lens.shape[0]."""
    c = cfg.c()
    _check(lib.mla_decode_step(ctypes.byref(c), _ptr(q_nope), _ptr(q_rope), _ptr(w_uk),
                               _ptr(ckv_raw), _ptr(krope_raw), _ptr(gamma), _ptr(seq_idx), _ptr(pos),
                               _ptr(block_table), int(block_table.shape[1]), _ptr(pool),
                               int(pool.shape[0]), _ptr(seq_lens), int(seq_lens.shape[0]),
                               q_per_seq, _ptr(q_work), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(out_latent),
                               _ptr(lse), _ptr(w_uv), _ptr(o), _ptr(dev_err), _stream(stream)),
           "mla_decode_step")


def output(cfg: Config, out_latent, w_uv, o, stream=None, dev_err=None):
    """mla_output: o[n, h] = W_UV[h] out_latent[n, h]."""
    c = cfg.c()
    _check(lib.mla_output(ctypes.byref(c), _ptr(out_latent), _ptr(w_uv), _ptr(o),
                          int(out_latent.shape[0]), _ptr(dev_err), _stream(stream)), "mla_output")


def combine_partials(cfg: Config, part_latent, part_lse, out_latent, lse=None, stream=None):
    """mla_combine_partials: merge part_latent (parts, n, H, r) / part_lse (parts, n, H), each
    part a decode over a disjoint set of the rows, into out_latent (n, H, r) and lse (n, H)."""
    c = cfg.c()
    _check(lib.mla_combine_partials(ctypes.byref(c), _ptr(part_latent), _ptr(part_lse),
                                    int(part_latent.shape[0]), int(part_latent.shape[1]),
                                    _ptr(out_latent), _ptr(lse), _stream(stream)),
           "mla_combine_partials")


def front_config(d_model: int, q_rank: int = 0, q_rms_eps: float = 1e-6) -> MlaFrontConfig:
    """mla_front_config: hidden size, query rank (0: full-rank query), RMSNorm eps of c_q."""
    return MlaFrontConfig(d_model, q_rank, q_rms_eps)


def project_workspace_size(cfg: Config, front: MlaFrontConfig, n_tokens: int) -> int:
    return int(lib.mla_project_workspace_size(ctypes.byref(cfg.c()), ctypes.byref(front),
                                              n_tokens))


def project(cfg: Config, front: MlaFrontConfig, x, w_dq, gamma_q, w_uq, w_qr, w_dkv, w_kr,
            q_nope, q_rope, ckv_raw, krope_raw, workspace, dev_err=None, stream=None):
    """mla_project: hidden states x (n, d_model) -> q_nope, q_rope, ckv_raw, krope_raw."""
    c = cfg.c()
    _check(lib.mla_project(ctypes.byref(c), ctypes.byref(front), _ptr(x), _ptr(w_dq),
                           _ptr(gamma_q), _ptr(w_uq), _ptr(w_qr), _ptr(w_dkv), _ptr(w_kr),
                           _ptr(q_nope), _ptr(q_rope), _ptr(ckv_raw), _ptr(krope_raw),
                           int(x.shape[0]), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _ptr(dev_err),
                           _stream(stream)), "mla_project")


def append_latent_fp8(cfg: Config, ckv_raw, krope_raw, gamma, seq_idx, pos, block_table, pool,
                      row_scale, dev_err, stream=None):
    """mla_append_latent_fp8: new rows as e4m3 codes (uint8 pool) with per-row scales."""
    c = cfg.c()
    _check(lib.mla_append_latent_fp8(ctypes.byref(c), _ptr(ckv_raw), _ptr(krope_raw), _ptr(gamma),
                                     _ptr(seq_idx), _ptr(pos), _ptr(block_table),
                                     int(block_table.shape[0]), int(block_table.shape[1]),
                                     _ptr(pool), _ptr(row_scale), int(pool.shape[0]),
                                     int(ckv_raw.shape[0]), _ptr(dev_err), _stream(stream)),
           "mla_append_latent_fp8")


def decode_fp8_workspace_size(cfg: Config, batch: int, q_per_seq: int, max_blocks: int) -> int:
    return int(lib.mla_decode_fp8_workspace_size(ctypes.byref(cfg.c()), batch, q_per_seq,
                                                 max_blocks))


def decode_fp8(cfg: Config, q, pool, row_scale, block_table, seq_lens, q_per_seq: int, workspace,
               out_latent, lse, dev_err, stream=None):
    """mla_decode_fp8: mla_decode over an fp8 pool (codes times the rows' scales)."""
    c = cfg.c()
    _check(lib.mla_decode_fp8(ctypes.byref(c), _ptr(q), _ptr(pool), _ptr(row_scale),
                              _ptr(block_table), int(block_table.shape[1]), int(pool.shape[0]),
                              _ptr(seq_lens), int(seq_lens.shape[0]), q_per_seq, _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(out_latent),
                              _ptr(lse), _ptr(dev_err), _stream(stream)), "mla_decode_fp8")


def prefill_workspace_size(cfg: Config, n_tokens: int) -> int:
    return int(lib.mla_prefill_workspace_size(ctypes.byref(cfg.c()), n_tokens))


def prefill(cfg: Config, q_nope, q_rope, pos, rows, w_uk, w_uv, cu_seqlens, max_seqlen: int, o,
            workspace, dev_err=None, stream=None):
    """mla_prefill: causal attention of packed prompts (cu_seqlens: batch + 1 offsets)."""
    c = cfg.c()
    _check(lib.mla_prefill(ctypes.byref(c), _ptr(q_nope), _ptr(q_rope), _ptr(pos), _ptr(rows),
                           _ptr(w_uk), _ptr(w_uv), _ptr(cu_seqlens), int(cu_seqlens.shape[0]) - 1,
                           int(max_seqlen), int(q_nope.shape[0]), _ptr(o), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _ptr(dev_err),
                           _stream(stream)), "mla_prefill")


# ---- speculative decoding with a drafted tree ------------------------------------------------
# These calls check what a raw pointer cannot carry (device, dtype, shape, contiguity) and raise
# MlaError before anything is launched; they launch on the tensors' device whichever device is
# current. The checks are written out in each call, and only a failed one asks _refuse which it
# was: a call of a few microseconds on the GPU should not take longer on the host.

torch = None  # imported by the first of these calls


def _import_torch():
    global torch
    import torch as module
    torch = module


def _refuse(where: str, device: int, *tensors):
    """Raise for the first (name, tensor, dtype, shape) that is not a contiguous tensor of that
    kind on GPU `device`."""
    for name, t, dtype, shape in tensors:
        if not t.is_cuda:
            raise MlaError(MLA_ERR_INVALID_ARG, f"{where}: {name} is on {t.device}, not on a GPU")
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device and
                t.is_contiguous()):
            continue
        raise MlaError(MLA_ERR_INVALID_ARG,
                       f"{where}: {name} is {t.dtype} {tuple(t.shape)} on {t.device}"
                       f"{'' if t.is_contiguous() else ' (not contiguous)'}, wanted {dtype} "
                       f"{tuple(shape)} on cuda:{device}")


def _sizes(where: str, name: str, t, dims: int):
    """The shape of a tensor whose sizes the call takes from it."""
    shape = t.shape
    if len(shape) != dims:
        raise MlaError(MLA_ERR_INVALID_ARG,
                       f"{where}: {name} has shape {tuple(shape)}, wanted {dims} dimensions")
    return shape


def _on(device: int, stream) -> int:
    """The raw handle of `stream`; None is the device's current one. (torch.cuda.current_stream()
    makes a Stream object, which takes longer than the rest of a small call.)"""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _elsewhere(where: str, device: int, fn, *args):
    """fn(*args) with `device` current, which it was not."""
    with torch.cuda.device(device):
        _check(fn(*args), where)


def build_tables(cfg: Config, seq_lens, new_lens, block_table, blocks_held, free_blocks,
                 free_count, blocks_held_out, free_count_out, cu_new, seq_idx, pos, slots, dev_err,
                 stream=None):
    """mla_build_tables: a step's block table and slot map from the requests' lengths.

    The pool has free_blocks.shape[0] blocks; blocks_held_out and free_count_out may be
    blocks_held and free_count.
    """
    if torch is None:
        _import_torch()
    w, i32 = "mla_build_tables", torch.int32
    dev = seq_lens.get_device()
    per, rows = _sizes(w, "seq_lens", seq_lens, 1), _sizes(w, "slots", slots, 1)
    blocks, width = _sizes(w, "free_blocks", free_blocks, 1)[0], _sizes(
        w, "block_table", block_table, 2)[1]
    n, tokens = per[0], rows[0]
    if not (seq_lens.is_cuda and seq_lens.dtype is i32 and seq_lens.is_contiguous() and
            new_lens.dtype is i32 and new_lens.shape == per and new_lens.get_device() == dev and
            new_lens.is_contiguous() and
            block_table.dtype is i32 and block_table.shape[0] == n and
            block_table.get_device() == dev and block_table.is_contiguous() and
            blocks_held.dtype is i32 and blocks_held.shape == per and
            blocks_held.get_device() == dev and blocks_held.is_contiguous() and
            free_blocks.dtype is i32 and free_blocks.get_device() == dev and
            free_blocks.is_contiguous() and
            free_count.dtype is i32 and free_count.shape == (1,) and
            free_count.get_device() == dev and
            blocks_held_out.dtype is i32 and blocks_held_out.shape == per and
            blocks_held_out.get_device() == dev and blocks_held_out.is_contiguous() and
            free_count_out.dtype is i32 and free_count_out.shape == (1,) and
            free_count_out.get_device() == dev and
            cu_new.dtype is i32 and cu_new.shape == (n + 1,) and cu_new.get_device() == dev and
            cu_new.is_contiguous() and
            seq_idx.dtype is i32 and seq_idx.shape == rows and seq_idx.get_device() == dev and
            seq_idx.is_contiguous() and
            pos.dtype is i32 and pos.shape == rows and pos.get_device() == dev and
            pos.is_contiguous() and
            slots.dtype is torch.int64 and slots.get_device() == dev and slots.is_contiguous() and
            dev_err.dtype is i32 and dev_err.shape == (1,) and dev_err.get_device() == dev):
        _refuse(w, dev, ("seq_lens", seq_lens, i32, (n,)), ("new_lens", new_lens, i32, (n,)),
                ("block_table", block_table, i32, (n, width)),
                ("blocks_held", blocks_held, i32, (n,)),
                ("free_blocks", free_blocks, i32, (blocks,)),
                ("free_count", free_count, i32, (1,)),
                ("blocks_held_out", blocks_held_out, i32, (n,)),
                ("free_count_out", free_count_out, i32, (1,)), ("cu_new", cu_new, i32, (n + 1,)),
                ("seq_idx", seq_idx, i32, (tokens,)), ("pos", pos, i32, (tokens,)),
                ("slots", slots, torch.int64, (tokens,)), ("dev_err", dev_err, i32, (1,)))
    args = (cfg.ref(), seq_lens.data_ptr(), new_lens.data_ptr(), n, block_table.data_ptr(), width,
            blocks_held.data_ptr(), free_blocks.data_ptr(), free_count.data_ptr(), blocks,
            blocks_held_out.data_ptr(), free_count_out.data_ptr(), cu_new.data_ptr(),
            seq_idx.data_ptr(), pos.data_ptr(), slots.data_ptr(), tokens, dev_err.data_ptr(),
            _on(dev, stream))
    if dev != torch._C._cuda_getDevice():
        return _elsewhere(w, dev, lib.mla_build_tables, *args)
    st = lib.mla_build_tables(*args)
    if st:
        raise MlaError(st, w)


def tree_masks(parents, seq_lens, mask, pos, dev_err, stream=None):
    """mla_tree_masks: ancestor masks (int32 words) and RoPE positions of drafted trees given by
    their parent indices, (batch, T), or (1, T) for one tree that all sequences share."""
    if torch is None:
        _import_torch()
    w, i32 = "mla_tree_masks", torch.int32
    dev = parents.get_device()
    n = _sizes(w, "seq_lens", seq_lens, 1)[0]
    rows, T = _sizes(w, "parents", parents, 2)
    if not (parents.is_cuda and parents.dtype is i32 and parents.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.get_device() == dev and seq_lens.is_contiguous() and
            mask.dtype is i32 and mask.shape == (n * T, (T + 31) // 32) and
            mask.get_device() == dev and mask.is_contiguous() and
            pos.dtype is i32 and pos.shape == (n * T,) and pos.get_device() == dev and
            pos.is_contiguous() and
            dev_err.dtype is i32 and dev_err.shape == (1,) and dev_err.get_device() == dev):
        _refuse(w, dev, ("parents", parents, i32, (rows, T)), ("seq_lens", seq_lens, i32, (n,)),
                ("mask", mask, i32, (n * T, (T + 31) // 32)), ("pos", pos, i32, (n * T,)),
                ("dev_err", dev_err, i32, (1,)))
    args = (parents.data_ptr(), rows, seq_lens.data_ptr(), n, T, mask.data_ptr(), pos.data_ptr(),
            dev_err.data_ptr(), _on(dev, stream))
    if dev != torch._C._cuda_getDevice():
        return _elsewhere(w, dev, lib.mla_tree_masks, *args)
    st = lib.mla_tree_masks(*args)
    if st:
        raise MlaError(st, w)


def append_slots(cfg: Config, ckv_raw, krope_raw, gamma, pos, slots, pool, dev_err, stream=None):
    """mla_append_slots: mla_append_latent's rows written to the pool rows `slots` (a negative
    slot is skipped), RoPE positions given apart. krope_raw may be None when rope_dim is 0."""
    if torch is None:
        _import_torch()
    w, dt, i32 = "mla_append_slots", cfg.torch_dtype, torch.int32
    dev = pool.get_device()
    per = _sizes(w, "slots", slots, 1)
    n, blocks, r, dr = per[0], _sizes(w, "pool", pool, 3)[0], cfg.kv_rank, cfg.rope_dim
    if not (pool.is_cuda and pool.dtype is dt and pool.is_contiguous() and
            pool.shape == (blocks, cfg.block_size, r + dr) and
            ckv_raw.dtype is dt and ckv_raw.shape == (n, r) and ckv_raw.get_device() == dev and
            ckv_raw.is_contiguous() and
            gamma.dtype is torch.float32 and gamma.shape == (r,) and gamma.get_device() == dev and
            gamma.is_contiguous() and
            pos.dtype is i32 and pos.shape == per and pos.get_device() == dev and
            pos.is_contiguous() and
            slots.dtype is torch.int64 and slots.get_device() == dev and slots.is_contiguous() and
            dev_err.dtype is i32 and dev_err.shape == (1,) and dev_err.get_device() == dev and
            (dr == 0 or (krope_raw.dtype is dt and krope_raw.shape == (n, dr) and
                         krope_raw.get_device() == dev and krope_raw.is_contiguous()))):
        _refuse(w, dev, ("pool", pool, dt, (blocks, cfg.block_size, r + dr)),
                ("ckv_raw", ckv_raw, dt, (n, r)), ("gamma", gamma, torch.float32, (r,)),
                ("pos", pos, i32, (n,)), ("slots", slots, torch.int64, (n,)),
                ("dev_err", dev_err, i32, (1,)),
                *([("krope_raw", krope_raw, dt, (n, dr))] if dr else []))
    args = (cfg.ref(), ckv_raw.data_ptr(), krope_raw.data_ptr() if dr else None, gamma.data_ptr(),
            pos.data_ptr(), slots.data_ptr(), pool.data_ptr(), blocks, n, dev_err.data_ptr(),
            _on(dev, stream))
    if dev != torch._C._cuda_getDevice():
        return _elsewhere(w, dev, lib.mla_append_slots, *args)
    st = lib.mla_append_slots(*args)
    if st:
        raise MlaError(st, w)


def decode_tree_workspace_size(cfg: Config, batch: int, q_per_seq: int) -> int:
    return int(lib.mla_decode_tree_workspace_size(cfg.ref(), batch, q_per_seq))


def decode_tree(cfg: Config, q, pool, block_table, seq_lens, q_per_seq: int, tree_mask, w_uv,
                workspace, o, lse, dev_err, stream=None):
    """mla_decode_tree: attention of every drafted token over its sequence's cache and the drafted
    rows its mask names (None: a chain), then W_UV. lse may be None."""
    if torch is None:
        _import_torch()
    w, dt, i32 = "mla_decode_tree", cfg.torch_dtype, torch.int32
    dev = pool.get_device()
    n = _sizes(w, "seq_lens", seq_lens, 1)[0]
    blocks, width = _sizes(w, "pool", pool, 3)[0], _sizes(w, "block_table", block_table, 2)[1]
    size = _sizes(w, "workspace", workspace, 1)[0]
    nt, H, r, bs = n * q_per_seq, cfg.num_heads, cfg.kv_rank, cfg.block_size
    D, dv = r + cfg.rope_dim, cfg.head_dim_v or cfg.head_dim
    if not (pool.is_cuda and pool.dtype is dt and pool.shape == (blocks, bs, D) and
            pool.is_contiguous() and
            q.dtype is dt and q.shape == (nt, H, D) and q.get_device() == dev and
            q.is_contiguous() and
            block_table.dtype is i32 and block_table.shape[0] == n and
            block_table.get_device() == dev and block_table.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.get_device() == dev and seq_lens.is_contiguous() and
            w_uv.dtype is dt and w_uv.shape == (H, dv, r) and w_uv.get_device() == dev and
            w_uv.is_contiguous() and
            workspace.dtype is torch.uint8 and workspace.get_device() == dev and
            workspace.is_contiguous() and
            o.dtype is dt and o.shape == (nt, H, dv) and o.get_device() == dev and
            o.is_contiguous() and
            dev_err.dtype is i32 and dev_err.shape == (1,) and dev_err.get_device() == dev and
            (tree_mask is None or
             (tree_mask.dtype is i32 and tree_mask.shape == (nt, (q_per_seq + 31) // 32) and
              tree_mask.get_device() == dev and tree_mask.is_contiguous())) and
            (lse is None or
             (lse.dtype is torch.float32 and lse.shape == (nt, H) and lse.get_device() == dev and
              lse.is_contiguous()))):
        _refuse(w, dev, ("pool", pool, dt, (blocks, bs, D)), ("q", q, dt, (nt, H, D)),
                ("block_table", block_table, i32, (n, width)), ("seq_lens", seq_lens, i32, (n,)),
                ("w_uv", w_uv, dt, (H, dv, r)), ("workspace", workspace, torch.uint8, (size,)),
                ("o", o, dt, (nt, H, dv)), ("dev_err", dev_err, i32, (1,)),
                *([] if tree_mask is None else
                  [("tree_mask", tree_mask, i32, (nt, (q_per_seq + 31) // 32))]),
                *([] if lse is None else [("lse", lse, torch.float32, (nt, H))]))
    args = (cfg.ref(), q.data_ptr(), pool.data_ptr(), block_table.data_ptr(), width, blocks,
            seq_lens.data_ptr(), n, q_per_seq, None if tree_mask is None else tree_mask.data_ptr(),
            w_uv.data_ptr(), workspace.data_ptr(), size, o.data_ptr(),
            None if lse is None else lse.data_ptr(), dev_err.data_ptr(), _on(dev, stream))
    if dev != torch._C._cuda_getDevice():
        return _elsewhere(w, dev, lib.mla_decode_tree, *args)
    st = lib.mla_decode_tree(*args)
    if st:
        raise MlaError(st, w)


def commit_tree(cfg: Config, path, path_len, q_per_seq: int, block_table, pool, seq_lens,
                seq_lens_out, dev_err, stream=None):
    """mla_commit_tree: the accepted path's rows moved together, seq_lens_out the lengths with it
    (may be seq_lens). path: (batch, width) node numbers, path_len of them count."""
    if torch is None:
        _import_torch()
    w, dt, i32 = "mla_commit_tree", cfg.torch_dtype, torch.int32
    dev = pool.get_device()
    per = _sizes(w, "seq_lens", seq_lens, 1)
    n, blocks, width = per[0], _sizes(w, "pool", pool, 3)[0], _sizes(
        w, "block_table", block_table, 2)[1]
    steps, D = _sizes(w, "path", path, 2)[1], cfg.kv_rank + cfg.rope_dim
    if not (pool.is_cuda and pool.dtype is dt and pool.shape == (blocks, cfg.block_size, D) and
            pool.is_contiguous() and
            path.dtype is i32 and path.shape[0] == n and path.get_device() == dev and
            path.is_contiguous() and
            path_len.dtype is i32 and path_len.shape == per and path_len.get_device() == dev and
            path_len.is_contiguous() and
            block_table.dtype is i32 and block_table.shape[0] == n and
            block_table.get_device() == dev and block_table.is_contiguous() and
            seq_lens.dtype is i32 and seq_lens.get_device() == dev and seq_lens.is_contiguous() and
            seq_lens_out.dtype is i32 and seq_lens_out.shape == per and
            seq_lens_out.get_device() == dev and seq_lens_out.is_contiguous() and
            dev_err.dtype is i32 and dev_err.shape == (1,) and dev_err.get_device() == dev):
        _refuse(w, dev, ("pool", pool, dt, (blocks, cfg.block_size, D)),
                ("path", path, i32, (n, steps)), ("path_len", path_len, i32, (n,)),
                ("block_table", block_table, i32, (n, width)), ("seq_lens", seq_lens, i32, (n,)),
                ("seq_lens_out", seq_lens_out, i32, (n,)), ("dev_err", dev_err, i32, (1,)))
    args = (cfg.ref(), path.data_ptr(), path_len.data_ptr(), steps, q_per_seq,
            block_table.data_ptr(), width, pool.data_ptr(), blocks, seq_lens.data_ptr(),
            seq_lens_out.data_ptr(), n, dev_err.data_ptr(), _on(dev, stream))
    if dev != torch._C._cuda_getDevice():
        return _elsewhere(w, dev, lib.mla_commit_tree, *args)
    st = lib.mla_commit_tree(*args)
    if st:
        raise MlaError(st, w)


def abi_version() -> int:
    return int(lib.mla_abi_version())
