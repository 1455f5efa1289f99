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

    def _held(self):
        # a struct is kept as long as the Config, so that no call's address outlives it, whatever
        # another thread does with the Config meanwhile
        key = (self.num_heads, self.head_dim, self.kv_rank, self.rope_dim, self.block_size,
               self.dtype, self.head_dim_v, self.rope_base, self.rms_eps, self.softmax_scale,
               self.decode_kernel)
        structs = self.__dict__.get("_structs")
        if structs is None:
            structs = self.__dict__.setdefault("_structs", {})
        held = structs.get(key)
        if held is None:
            c = self.c()
            held = structs.setdefault(key, (c, ctypes.byref(c), ctypes.addressof(c)))
        return held

    def __getstate__(self):  # copies and pickles without the structs
        return {k: v for k, v in self.__dict__.items() if k != "_structs"}

    def ref(self):
        """A reference to the C struct for a call; built again only when a field has changed."""
        return self._held()[1]

    def address(self) -> int:
        """The address of that struct."""
        return self._held()[2]

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
# current. Checks and call are in a compiled module (csrc/fast_call.cpp): a call of a few
# microseconds on the GPU should not take longer on the host. _refuse says what it refused.

class _Fast:
    """The compiled module, loaded on first use and given the library's functions."""

    def __getattr__(self, name):
        import torch  # noqa: F401  (its libraries are the module's)
        try:
            from . import _fast_call
        except ImportError as e:
            raise ImportError("mla_latent_kv_44_b200/_fast_call.so cannot be loaded: build it with "
                              f"`python -m mla_latent_kv_44_b200.build` ({e})") from e
        for call in ("build_tables", "tree_masks", "append_slots", "decode_tree", "commit_tree"):
            fn = getattr(lib, "mla_" + call)
            _fast_call.bind("mla_" + call, ctypes.cast(fn, _vp).value)
            self.__dict__[call] = getattr(_fast_call, call)
        return self.__dict__[name]


_fast = _Fast()


def _raw(stream):
    """None (the current stream of the tensors' device) or the handle of a stream."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _refuse(where: str, *tensors):
    """Raise for the first (name, tensor, dtype, shape) that is not a contiguous tensor of that
    kind on the first one's GPU. A None in a shape stands for any size."""
    import torch
    device = None
    for name, t, dtype, shape in tensors:
        if not isinstance(t, torch.Tensor):
            raise MlaError(MLA_ERR_INVALID_ARG,
                           f"{where}: {name} is {type(t).__name__}, not a tensor")
        if t.dim() != len(shape):
            raise MlaError(MLA_ERR_INVALID_ARG, f"{where}: {name} has shape {tuple(t.shape)}, "
                           f"wanted {len(shape)} dimensions")
        if not t.is_cuda:
            raise MlaError(MLA_ERR_INVALID_ARG, f"{where}: {name} is on {t.device}, not on a GPU")
        device = t.device if device is None else device
        if (t.dtype is dtype and t.device == device and t.is_contiguous() and
                all(w is None or w == n for n, w in zip(t.shape, shape))):
            continue
        raise MlaError(MLA_ERR_INVALID_ARG,
                       f"{where}: {name} is {t.dtype} {tuple(t.shape)} on {t.device}"
                       f"{'' if t.is_contiguous() else ' (not contiguous)'}, wanted {dtype} "
                       f"({', '.join('any' if n is None else str(n) for n in shape)}) on {device}")
    raise MlaError(MLA_ERR_INVALID_ARG, where)


def _size(t, dim: int):
    """A size that the other tensors' shapes follow; None where t has no such dimension."""
    return t.shape[dim] if getattr(t, "ndim", 0) > dim else None


def _finish(where: str, st: int, first, call, args, tensors):
    """What is left to do when a fast call did not return MLA_OK."""
    if st == -2:  # the tensors are on another device than the current one
        import torch
        with torch.cuda.device(first.device):
            st = call(*args)
    if st == -1:
        _refuse(where, *tensors())
    _check(st, where)


def build_tables(cfg: Config, seq_lens, new_lens, block_table, blocks_held, free_blocks,
                 free_count, blocks_held_out, free_count_out, cu_new, seq_idx, pos, slots, dev_err,
                 stream=None):
    """mla_build_tables: a step's block table and slot map from the requests' lengths.

    The pool has free_blocks.shape[0] blocks; blocks_held_out and free_count_out may be
    blocks_held and free_count.
    """
    args = (cfg.address(), seq_lens, new_lens, block_table, blocks_held, free_blocks, free_count,
            blocks_held_out, free_count_out, cu_new, seq_idx, pos, slots, dev_err, _raw(stream))
    st = _fast.build_tables(*args)
    if st:
        def tensors():
            import torch
            i32, n, m = torch.int32, _size(seq_lens, 0), _size(slots, 0)
            return (("seq_lens", seq_lens, i32, (n,)), ("new_lens", new_lens, i32, (n,)),
                    ("block_table", block_table, i32, (n, None)),
                    ("blocks_held", blocks_held, i32, (n,)),
                    ("free_blocks", free_blocks, i32, (None,)),
                    ("free_count", free_count, i32, (1,)),
                    ("blocks_held_out", blocks_held_out, i32, (n,)),
                    ("free_count_out", free_count_out, i32, (1,)),
                    ("cu_new", cu_new, i32, (None if n is None else n + 1,)),
                    ("seq_idx", seq_idx, i32, (m,)), ("pos", pos, i32, (m,)),
                    ("slots", slots, torch.int64, (m,)), ("dev_err", dev_err, i32, (1,)))
        _finish("mla_build_tables", st, seq_lens, _fast.build_tables, args, tensors)


def tree_masks(parents, seq_lens, mask, pos, dev_err, stream=None):
    """mla_tree_masks: ancestor masks (int32 words) and RoPE positions of drafted trees given by
    their parent indices, (batch, T), or (1, T) for one tree that all sequences share."""
    args = (parents, seq_lens, mask, pos, dev_err, _raw(stream))
    st = _fast.tree_masks(*args)
    if st:
        def tensors():
            import torch
            i32, n, T = torch.int32, _size(seq_lens, 0), _size(parents, 1)
            m = None if n is None or T is None else n * T
            return (("parents", parents, i32, (None, T)), ("seq_lens", seq_lens, i32, (n,)),
                    ("mask", mask, i32, (m, None if T is None else (T + 31) // 32)),
                    ("pos", pos, i32, (m,)), ("dev_err", dev_err, i32, (1,)))
        _finish("mla_tree_masks", st, parents, _fast.tree_masks, args, tensors)


def append_slots(cfg: Config, ckv_raw, krope_raw, gamma, pos, slots, pool, dev_err, stream=None):
    """mla_append_slots: mla_append_latent's rows written to the pool rows `slots` (a negative
    slot is skipped), RoPE positions given apart. krope_raw may be None when rope_dim is 0."""
    args = (cfg.address(), ckv_raw, krope_raw, gamma, pos, slots, pool, dev_err, _raw(stream))
    st = _fast.append_slots(*args)
    if st:
        def tensors():
            import torch
            dt, n, r, dr = cfg.torch_dtype, _size(slots, 0), cfg.kv_rank, cfg.rope_dim
            return (("pool", pool, dt, (None, cfg.block_size, r + dr)),
                    ("ckv_raw", ckv_raw, dt, (n, r)), ("gamma", gamma, torch.float32, (r,)),
                    ("pos", pos, torch.int32, (n,)), ("slots", slots, torch.int64, (n,)),
                    ("dev_err", dev_err, torch.int32, (1,)),
                    *((("krope_raw", krope_raw, dt, (n, dr)),) if dr else ()))
        _finish("mla_append_slots", st, pool, _fast.append_slots, args, tensors)


def decode_tree_workspace_size(cfg: Config, batch: int, q_per_seq: int) -> int:
    if not (0 < batch < 1 << 31 and 0 < q_per_seq < 1 << 31):  # ctypes takes numbers modulo 2^32
        return 0
    return int(lib.mla_decode_tree_workspace_size(cfg.ref(), batch, q_per_seq))


def decode_tree(cfg: Config, q, pool, block_table, seq_lens, q_per_seq: int, tree_mask, w_uv,
                workspace, o, lse, dev_err, stream=None):
    """mla_decode_tree: attention of every drafted token over its sequence's cache and the drafted
    rows its mask names (None: a chain), then W_UV. lse may be None."""
    args = (cfg.address(), q, pool, block_table, seq_lens, q_per_seq, tree_mask, w_uv, workspace, o,
            lse, dev_err, _raw(stream))
    st = _fast.decode_tree(*args)
    if st:
        def tensors():
            import torch
            dt, i32, n = cfg.torch_dtype, torch.int32, _size(seq_lens, 0)
            nt = None if n is None else n * q_per_seq
            H, r, dv = cfg.num_heads, cfg.kv_rank, cfg.head_dim_v or cfg.head_dim
            return (("pool", pool, dt, (None, cfg.block_size, r + cfg.rope_dim)),
                    ("q", q, dt, (nt, H, r + cfg.rope_dim)),
                    ("block_table", block_table, i32, (n, None)),
                    ("seq_lens", seq_lens, i32, (n,)), ("w_uv", w_uv, dt, (H, dv, r)),
                    ("workspace", workspace, torch.uint8, (None,)), ("o", o, dt, (nt, H, dv)),
                    ("dev_err", dev_err, i32, (1,)),
                    *(() if tree_mask is None else
                      (("tree_mask", tree_mask, i32, (nt, (q_per_seq + 31) // 32)),)),
                    *(() if lse is None else (("lse", lse, torch.float32, (nt, H)),)))
        _finish("mla_decode_tree", st, pool, _fast.decode_tree, args, tensors)


def commit_tree(cfg: Config, path, path_len, q_per_seq: int, block_table, pool, seq_lens,
                seq_lens_out, dev_err, stream=None):
    """mla_commit_tree: the accepted path's rows moved together, seq_lens_out the lengths with it
    (may be seq_lens). path: (batch, width) node numbers, path_len of them count."""
    args = (cfg.address(), path, path_len, q_per_seq, block_table, pool, seq_lens, seq_lens_out,
            dev_err, _raw(stream))
    st = _fast.commit_tree(*args)
    if st:
        def tensors():
            import torch
            i32, n = torch.int32, _size(seq_lens, 0)
            return (("pool", pool, cfg.torch_dtype,
                     (None, cfg.block_size, cfg.kv_rank + cfg.rope_dim)),
                    ("path", path, i32, (n, None)), ("path_len", path_len, i32, (n,)),
                    ("block_table", block_table, i32, (n, None)),
                    ("seq_lens", seq_lens, i32, (n,)), ("seq_lens_out", seq_lens_out, i32, (n,)),
                    ("dev_err", dev_err, i32, (1,)))
        _finish("mla_commit_tree", st, pool, _fast.commit_tree, args, tensors)


def abi_version() -> int:
    return int(lib.mla_abi_version())
