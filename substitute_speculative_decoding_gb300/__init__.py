"""Python binding of the SubSpec CUDA library (libsubspec.so, sm_103a).

Argument marshalling only: every step of the decode path runs in the
library's kernels.  PyTorch provides device memory, pinned host memory and
streams.  There is no CPU fallback: importing this package fails loudly when
the library has not been built (run ``substitute_speculative_decoding_gb300/build.py``
or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes as C
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsubspec.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build the CUDA library first "
                      "(python substitute_speculative_decoding_gb300/build.py)")
_lib = C.CDLL(LIB_PATH)

SUB_OK, SUB_EINVAL, SUB_ENOMEM, SUB_ECUDA, SUB_EUNSUPPORTED, SUB_ETIMEOUT = range(6)
_NAMES = {1: "EINVAL", 2: "ENOMEM", 3: "ECUDA", 4: "EUNSUPPORTED", 5: "ETIMEOUT"}


class SubError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"SUB_{_NAMES.get(code, code)}: {msg}")
        self.code = code


_vp = C.c_void_p
_i32, _i64, _u64, _f32 = C.c_int32, C.c_int64, C.c_uint64, C.c_float


class KVCache(C.Structure):
    """sub_kv_cache.  device: where its tensors are; n_seqs: rows of its page table."""
    device, n_seqs = None, 1
    _fields_ = [("k", _vp), ("v", _vp), ("page_table", _vp), ("n_layers", _i32),
                ("n_heads_kv", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("n_pages", _i32), ("capacity", _i64)]


class KV8Cache(C.Structure):
    """sub_kv8_cache, with the same."""
    device, n_seqs = None, 1
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_table", _vp),
                ("n_layers", _i32), ("n_heads_kv", _i32), ("head_dim", _i32),
                ("page_size", _i32), ("n_pages", _i32), ("capacity", _i64)]


class Batch(C.Structure):
    _fields_ = [("start", _vp), ("pos", _vp), ("n_seqs", _i32), ("n_rows", _i32),
                ("max_keys", _i64)]


class Rope(C.Structure):
    """sub_rope: the rotation of position embeddings."""
    _fields_ = [("step", _u64 * 64), ("head_dim", _i32)]


class Tree(C.Structure):
    _fields_ = [("token", _vp), ("parent", _vp), ("depth", _vp), ("score", _vp), ("anc", _vp),
                ("width", _i32), ("max_depth", _i32)]


class W4(C.Structure):
    _fields_ = [("q", _vp), ("scale", _vp), ("zero", _vp), ("bits", _i32)]


class LayerDesc(C.Structure):
    _fields_ = [(n, _vp) for n in ("wq", "wk", "wv", "wo", "wg", "wu", "wd",
                                   "attn_norm", "ffn_norm")] + \
               [(n, W4) for n in ("q4", "k4", "v4", "o4", "g4", "u4", "d4")]


class ModelDesc(C.Structure):
    _fields_ = [(n, _i32) for n in ("n_layers", "hidden", "n_heads_q", "n_heads_kv", "head_dim",
                                    "ffn", "vocab", "n_resident")] + \
               [("rope_theta", _f32), ("rms_eps", _f32), ("embed", _vp), ("lm_head", _vp),
                ("final_norm", _vp), ("layers", C.POINTER(LayerDesc))] + \
               [(n, _i32) for n in ("max_seq", "max_depth", "max_width", "staging_layers",
                                    "max_prompt")]


class DecodeCfg(C.Structure):
    _fields_ = [("depth", _i32), ("width", _i32), ("draft_temp", _f32), ("mode", _i32),
                ("target_temp", _f32), ("seed", _u64), ("use_graph", _i32),
                ("stop_logp", _f32), ("verify_reuse", _i32)]


class Stats(C.Structure):
    _fields_ = [("cycles", _i64), ("emitted", _i64), ("tau", C.c_double),
                ("t_prefill_ms", C.c_double), ("t_decode_ms", C.c_double),
                ("accept_hist", _i64 * 65), ("t_draft_ms", C.c_double),
                ("t_verify_ms", C.c_double), ("t_copy_unhidden_ms", C.c_double),
                ("near_tie_events", _i64), ("drafted_levels", _i64), ("t_copy_ms", C.c_double)]


def _decl(name, args):
    f = getattr(_lib, name)
    f.argtypes = args
    f.restype = _i32
    return f


_lib.sub_last_error.restype = C.c_char_p
_lib.sub_last_error.argtypes = []
_lib.sub_version.restype = C.c_char_p
_lib.sub_version.argtypes = []
_pipeline_timeouts = _decl("sub_pipeline_timeouts", [_vp])
_bounded_wait_check = _decl("sub_bounded_wait_check", [C.c_uint32])

_w4_pack = _decl("sub_w4_pack", [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp])
_w4_dequant = _decl("sub_w4_dequant", [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp])
_w4_gemm = _decl("sub_w4_gemm", [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp])
_bf16_gemm = _decl("sub_bf16_gemm", [_vp, _i64, _vp, _i64, _i64, _vp, _vp])
_wq_pack = _decl("sub_wq_pack", [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp])
_wq_dequant = _decl("sub_wq_dequant", [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp])
_wq_pack_hqq = _decl("sub_wq_pack_hqq", [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp])
_wq_gemm = _decl("sub_wq_gemm", [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp])
_tree_attn = _decl("sub_tree_attn", [_vp, _i32, _i32, C.POINTER(KVCache), _i32, _i64, _i64, _i32,
                                     _vp, _i32, _vp, _f32, _vp, _vp])
_draft_expand = _decl("sub_draft_expand", [_vp, _i64, _f32, C.POINTER(Tree), _i32, _vp])
_verify_accept = _decl("sub_verify_accept", [_vp, C.POINTER(Tree), _i32, _i64, _i32, _f32, _u64,
                                             _i64, _vp, _vp, _vp, _vp, _vp])
_verify_accept_static = _decl("sub_verify_accept_static",
                              [_vp, C.POINTER(Tree), _i32, _i64, _i32, _f32, _u64, _i64, _vp, _vp,
                               _vp, _vp, _vp])
_kv_compact = _decl("sub_kv_compact", [C.POINTER(KVCache), _i64, _vp, _vp, _i32, _vp])
_KV, _KV8, _BATCH = C.POINTER(KVCache), C.POINTER(KV8Cache), C.POINTER(Batch)
_kv_append = _decl("sub_kv_append", [_vp, _i64, _vp, _i64, _KV, _i32, _BATCH, _vp])
_kv8_append = _decl("sub_kv8_append", [_vp, _i64, _vp, _i64, _KV8, _i32, _BATCH, _vp])
_kv8_read = _decl("sub_kv8_read", [_KV8, _i32, _BATCH, _vp, _vp, _vp])
_chunk_attn = _decl("sub_chunk_attn", [_vp, _i64, _i32, _KV, _i32, _BATCH, _f32, _vp, _vp, _i64,
                                       _vp])
_chunk_attn8 = _decl("sub_chunk_attn8", [_vp, _i64, _i32, _KV8, _i32, _BATCH, _f32, _vp, _vp,
                                         _i64, _vp])
_chunk_attn_workspace = _decl("sub_chunk_attn_workspace", [_i32, _i32, _i32, _i32, _i32,
                                                           C.POINTER(_i64)])
_ROPE = C.POINTER(Rope)
_rope_init = _decl("sub_rope_init", [_i32, C.c_double, C.POINTER(C.c_double), _ROPE])
_kv_append_rope = _decl("sub_kv_append_rope", [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _KV, _i32,
                                               _BATCH, _ROPE, _vp, _vp, _i64, _vp])
_kv8_append_rope = _decl("sub_kv8_append_rope", [_vp, _i64, _i32, _vp, _i64, _vp, _i64, _KV8, _i32,
                                                 _BATCH, _ROPE, _vp, _vp, _i64, _vp])
_kv_move = _decl("sub_kv_move", [_KV, _i32, _vp, _vp, _i32, _vp, _vp])
_kv8_move = _decl("sub_kv8_move", [_KV8, _i32, _vp, _vp, _i32, _vp, _vp])
_chunk_tree_attn = _decl("sub_chunk_tree_attn", [_vp, _i64, _i32, _KV, _i32, _BATCH, _vp, _vp, _i32,
                                                 _f32, _vp, _vp, _i64, _vp])
_chunk_tree_attn8 = _decl("sub_chunk_tree_attn8", [_vp, _i64, _i32, _KV8, _i32, _BATCH, _vp, _vp,
                                                   _i32, _f32, _vp, _vp, _i64, _vp])
_beam_select = _decl("sub_beam_select", [_vp, _vp, _i32, _i32, _i64, _f32, _i32, _vp, _i32, _i32,
                                         _vp, _vp, _vp, _vp, _vp, _i64, _vp])
_beam_workspace = _decl("sub_beam_workspace", [_i32, _i32, _i64, C.POINTER(_i64)])
_probs = _decl("sub_probs", [_vp, _i64, _i64, _f32, _vp, _vp])
_verify_sample = _decl("sub_verify_sample", [_vp, _vp, _vp, _vp, _i32, _i32, _i64, _vp, _vp, _vp])
_model_create = _decl("sub_model_create", [C.POINTER(ModelDesc), C.POINTER(_vp)])
_model_destroy = _decl("sub_model_destroy", [_vp])
_model_memory = _decl("sub_model_memory", [_vp, C.POINTER(_i64)])
_model_forward = _decl("sub_model_forward", [_vp, _i32, _vp, _i32, _i32, _vp, _vp, _i32, _i64,
                                             _vp, _vp])
_model_kv = _decl("sub_model_kv", [_vp, C.POINTER(KVCache)])
_generate = _decl("sub_generate", [_vp, _vp, _i32, _i32, C.POINTER(DecodeCfg), _vp,
                                   C.POINTER(Stats)])
_prefill = _decl("sub_prefill", [_vp, _vp, _i32, C.POINTER(DecodeCfg), _vp])
_decode_cycles = _decl("sub_decode_cycles", [_vp, C.POINTER(DecodeCfg), _i32, _vp])
_decode_read = _decl("sub_decode_read", [_vp, _vp, _i32, C.POINTER(_i32), C.POINTER(_i64)])
_cycle_info = _decl("sub_cycle_info", [_vp, C.POINTER(DecodeCfg), C.POINTER(_i64),
                                       C.POINTER(_i64)])

EXPORTED = ["sub_last_error", "sub_version", "sub_pipeline_timeouts", "sub_bounded_wait_check",
            "sub_w4_pack", "sub_w4_dequant", "sub_w4_gemm",
            "sub_wq_pack", "sub_wq_dequant", "sub_wq_gemm", "sub_wq_pack_hqq",
            "sub_bf16_gemm", "sub_tree_attn", "sub_draft_expand", "sub_verify_accept",
            "sub_verify_accept_static",
            "sub_kv_compact", "sub_kv_append", "sub_kv8_append", "sub_kv8_read", "sub_chunk_attn",
            "sub_chunk_attn8", "sub_chunk_attn_workspace", "sub_rope_init",
            "sub_kv_append_rope", "sub_kv8_append_rope", "sub_kv_move", "sub_kv8_move",
            "sub_chunk_tree_attn", "sub_chunk_tree_attn8", "sub_beam_select", "sub_beam_workspace",
            "sub_probs", "sub_verify_sample",
            "sub_model_create", "sub_model_destroy", "sub_model_memory",
            "sub_model_forward", "sub_model_kv", "sub_generate", "sub_prefill",
            "sub_decode_cycles", "sub_decode_read", "sub_cycle_info"]


def _check(code):
    if code != SUB_OK:
        raise SubError(code, _lib.sub_last_error().decode())


def version() -> str:
    return _lib.sub_version().decode()


def pipeline_timeouts() -> int:
    """Bounded pipeline waits that ran out on this device (0 in a correct run)."""
    n = C.c_uint32(0)
    _check(_pipeline_timeouts(C.byref(n)))
    return int(n.value)


def bounded_wait_check(max_polls: int) -> int:
    """Run the bounded-wait check kernel; returns its status code
    (SUB_ETIMEOUT when the wait gave up, as it must)."""
    return int(_bounded_wait_check(max_polls))


def _p(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _bf16(t):
    assert t.dtype == torch.bfloat16 and t.is_contiguous()
    return t


# ------------------------------------------------------------------ kernels --
def w4_pack(w: torch.Tensor, stream=None):
    """Group-64 min-max int4 pack of a bf16 [N, K] device matrix -> (q, scale, zero)."""
    n, k = w.shape
    g = (k + 63) // 64
    q = torch.empty((n, g * 32), dtype=torch.uint8, device=w.device)
    s = torch.empty((n, g), dtype=torch.bfloat16, device=w.device)
    z = torch.empty((n, g), dtype=torch.bfloat16, device=w.device)
    _check(_w4_pack(_p(_bf16(w)), n, k, 64, _p(q), _p(s), _p(z), _stream(stream)))
    return q, s, z


def w4_dequant(q, s, z, k: int, stream=None):
    n = q.shape[0]
    out = torch.empty((n, k), dtype=torch.bfloat16, device=q.device)
    _check(_w4_dequant(_p(q), _p(s), _p(z), n, k, 64, _p(out), _stream(stream)))
    return out


def w4_gemm(x, q, s, z, n: int, k: int, out=None, stream=None):
    m = x.shape[0]
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _check(_w4_gemm(_p(_bf16(x)), m, _p(q), _p(s), _p(z), n, k, 64, _p(y), _stream(stream)))
    return y


def wq_pack(w: torch.Tensor, bits: int, stream=None):
    """Group-64 min-max pack with 2, 3 or 4 code bits of a bf16 [N, K] device
    matrix -> (q uint8 [N, G * 8 * bits], scale, zero)."""
    n, k = w.shape
    g = (k + 63) // 64
    q = torch.empty((n, g * 8 * bits), dtype=torch.uint8, device=w.device)
    s = torch.empty((n, g), dtype=torch.bfloat16, device=w.device)
    z = torch.empty((n, g), dtype=torch.bfloat16, device=w.device)
    _check(_wq_pack(_p(_bf16(w)), n, k, 64, bits, _p(q), _p(s), _p(z), _stream(stream)))
    return q, s, z


def wq_pack_hqq(w: torch.Tensor, bits: int, iters: int = 20, stream=None):
    """wq_pack with the HQQ-optimised zero point -> (q, scale, zero)."""
    n, k = w.shape
    g = (k + 63) // 64
    q = torch.empty((n, g * 8 * bits), dtype=torch.uint8, device=w.device)
    s = torch.empty((n, g), dtype=torch.bfloat16, device=w.device)
    z = torch.empty((n, g), dtype=torch.bfloat16, device=w.device)
    _check(_wq_pack_hqq(_p(_bf16(w)), n, k, 64, bits, iters, _p(q), _p(s), _p(z),
                        _stream(stream)))
    return q, s, z


def wq_dequant(q, s, z, k: int, bits: int, stream=None):
    n = q.shape[0]
    out = torch.empty((n, k), dtype=torch.bfloat16, device=q.device)
    _check(_wq_dequant(_p(q), _p(s), _p(z), n, k, 64, bits, _p(out), _stream(stream)))
    return out


def wq_gemm(x, q, s, z, n: int, k: int, bits: int, out=None, stream=None):
    m = x.shape[0]
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _check(_wq_gemm(_p(_bf16(x)), m, _p(q), _p(s), _p(z), n, k, 64, bits, _p(y),
                    _stream(stream)))
    return y


def bf16_gemm(x, w, out=None, stream=None):
    m, k = x.shape
    n = w.shape[0]
    y = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _check(_bf16_gemm(_p(_bf16(x)), m, _p(_bf16(w)), n, k, _p(y), _stream(stream)))
    return y


def tree_attn(q, kv: KVCache, layer: int, n_prefix: int, tree_base: int, n_slots: int,
              anc=None, depth=None, scale=None, out=None, stream=None):
    n_q, hq, d = q.shape
    o = out if out is not None else torch.empty_like(q)
    scale = scale if scale is not None else d ** -0.5
    _check(_tree_attn(_p(_bf16(q)), n_q, hq, C.byref(kv), layer, n_prefix, tree_base, n_slots,
                      _p(anc), 0 if anc is None else anc.shape[1], _p(depth), scale, _p(o),
                      _stream(stream)))
    return o


class DeviceTree:
    """Device arrays of a static tree with 1 + depth*width slots."""

    def __init__(self, depth: int, width: int, device="cuda"):
        n = 1 + depth * width
        self.depth_max, self.width = depth, width
        self.token = torch.zeros(n, dtype=torch.int32, device=device)
        self.parent = torch.full((n,), -1, dtype=torch.int32, device=device)
        self.depth = torch.zeros(n, dtype=torch.int32, device=device)
        self.score = torch.zeros(n, dtype=torch.float32, device=device)
        self.anc = torch.full((n, depth + 1), -1, dtype=torch.int32, device=device)
        self.anc[0, 0] = 0

    def struct(self) -> Tree:
        return Tree(self.token.data_ptr(), self.parent.data_ptr(), self.depth.data_ptr(),
                    self.score.data_ptr(), self.anc.data_ptr(), self.width, self.depth_max)


def draft_expand(logits, temperature: float, tree: DeviceTree, level: int, stream=None):
    t = tree.struct()
    _check(_draft_expand(_p(logits), logits.shape[1], temperature, C.byref(t), level,
                         _stream(stream)))


def verify_accept(logits, tree: DeviceTree, n_nodes: int, mode=0, temperature=1.0, seed=0,
                  root_pos=0, stream=None, out=None, with_choice=True):
    """Returns device tensors (accepted slots [D], n_accepted [1], bonus [1],
    choice [n] or None).  `out` reuses those four tensors."""
    return _accept(_verify_accept, logits, tree, n_nodes, mode, temperature, seed, root_pos,
                   stream, out, with_choice)


def verify_accept_static(logits, tree: DeviceTree, n_nodes: int, mode=0, temperature=1.0,
                         seed=0, root_pos=0, stream=None, out=None, with_choice=True):
    """verify_accept on the library's fixed per-device scratch (no device
    allocation inside the call; calls on one device must be ordered)."""
    return _accept(_verify_accept_static, logits, tree, n_nodes, mode, temperature, seed,
                   root_pos, stream, out, with_choice)


def _accept(fn, logits, tree, n_nodes, mode, temperature, seed, root_pos, stream, out,
            with_choice):
    dev = logits.device
    if out is None:
        out = (torch.zeros(max(tree.depth_max, 1), dtype=torch.int32, device=dev),
               torch.zeros(1, dtype=torch.int32, device=dev),
               torch.zeros(1, dtype=torch.int32, device=dev),
               torch.zeros(n_nodes, dtype=torch.int32, device=dev) if with_choice else None)
    acc, na, bonus, choice = out
    t = tree.struct()
    _check(fn(_p(logits), C.byref(t), n_nodes, logits.shape[1], mode, temperature, seed, root_pos,
              _p(acc), _p(na), _p(bonus), _p(choice),
              _stream(stream)))
    return acc, na, bonus, choice


def kv_compact(kv: KVCache, root_pos: int, accepted, n_accepted, max_accept: int, stream=None):
    _check(_kv_compact(C.byref(kv), root_pos, _p(accepted), _p(n_accepted), max_accept,
                       _stream(stream)))


def make_kv(n_layers, n_heads_kv, head_dim, capacity, page_size=64, device="cuda",
            shuffle_seed=None):
    """A paged cache owned by torch tensors (pages optionally permuted)."""
    n_pages = (capacity + page_size - 1) // page_size
    k = torch.zeros((n_layers, n_pages, n_heads_kv, page_size, head_dim), dtype=torch.bfloat16,
                    device=device)
    v = torch.zeros_like(k)
    if shuffle_seed is None:
        pt = torch.arange(n_pages, dtype=torch.int32)
    else:
        pt = torch.randperm(n_pages, generator=torch.Generator().manual_seed(shuffle_seed))
        pt = pt.to(torch.int32)
    pt = pt.to(device)
    st = KVCache(k.data_ptr(), v.data_ptr(), pt.data_ptr(), n_layers, n_heads_kv, head_dim,
                 page_size, n_pages, n_pages * page_size)
    st.device = k.device
    return st, (k, v, pt)


# ----------------------------------------------- batches of sequences --
# These calls are made once per layer or token, so their checks cost little on
# the way that is taken: messages are formed only when one fails.
def _refuse(msg):
    raise SubError(SUB_EINVAL, msg)


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name}: a tensor on the GPU is needed")
    return t.device


def _dense(t, dtype, shape, name, device):
    """Address of a contiguous tensor of this type and shape on the device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        _refuse(f"{name}: must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _rows(t, rows, heads, d, name, device):
    """Row stride of a bf16 tensor [rows, heads, d] whose rows may lie apart."""
    if t.dtype is not torch.bfloat16 or t.shape != (rows, heads, d) or t.device != device:
        _refuse(f"{name}: must be a bf16 tensor of shape {(rows, heads, d)} on {device}")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d > 1) or (s1 != d and heads > 1):
        _refuse(f"{name}: the heads of a row must be contiguous")
    return s0 if rows > 1 else heads * d


def _new(shape, dtype, device, stream, zero):
    """A tensor allocated (and zeroed) on the call's stream."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _run(fn, device, stream, *args):
    """The library's call on the tensors' device, on the given or current stream."""
    i = device.index
    if torch._C._cuda_getDevice() != i:
        with torch.cuda.device(i):
            return _run(fn, device, stream, *args)
    code = fn(*args, torch._C._cuda_getCurrentRawStream(i) if stream is None
              else stream.cuda_stream)
    if code != SUB_OK:
        _check(code)


def _run_scratch(fn, device, stream, size, *args):
    """_run with `size` bytes of workspace that the call's stream has to itself, as the last
    arguments.  From torch's allocator without a tensor around it: among driver calls
    torch.empty costs the host 5 us, this 2."""
    i = device.index
    if torch._C._cuda_getDevice() != i:
        with torch.cuda.device(i):
            return _run_scratch(fn, device, stream, size, *args)
    if size == 0:
        return _run(fn, device, stream, *args, None, 0)
    st = torch._C._cuda_getCurrentRawStream(i) if stream is None else stream.cuda_stream
    p = torch._C._cuda_cudaCachingAllocator_raw_alloc(size, st)
    try:
        code = fn(*args, p, size, st)
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(p)
    if code != SUB_OK:
        _check(code)


def _paged(struct, dtype, k, v, page_table, scales=()):
    dev = _gpu(k, "k")
    if k.dim() != 5:
        _refuse("k: must be [n_layers, n_pages, n_heads_kv, page_size, head_dim]")
    if page_table.dim() != 2 or page_table.shape[1] < 1:
        _refuse("page_table: must be [n_seqs, pages per sequence]")
    shape = k.shape
    nl, npg, h, ps, d = shape
    at = [_dense(k, dtype, shape, "k", dev), _dense(v, dtype, shape, "v", dev)]
    at += [_dense(x, torch.float32, shape[:4], n, dev) for x, n in scales]
    at.append(_dense(page_table, torch.int32, page_table.shape, "page_table", dev))
    kv = struct(*at, nl, h, d, ps, npg, page_table.shape[1] * ps)
    kv.keep = (k, v, page_table, *(x for x, _ in scales))
    kv.device, kv.n_seqs = dev, page_table.shape[0]
    return kv


def paged_kv(k, v, page_table) -> KVCache:
    """A cache of sequences on torch tensors: pools k, v bf16 [n_layers, n_pages,
    n_heads_kv, page_size, head_dim], page_table int32 [n_seqs, pages per
    sequence] (entries outside the pool: no page).  Keeps the tensors."""
    return _paged(KVCache, torch.bfloat16, k, v, page_table)


def paged_kv8(k, v, k_scale, v_scale, page_table) -> KV8Cache:
    """An 8-bit cache of sequences: codes uint8 shaped as paged_kv's pools, scales
    fp32 without the last axis."""
    return _paged(KV8Cache, torch.uint8, k, v, page_table,
                  ((k_scale, "k_scale"), (v_scale, "v_scale")))


def batch(start, pos, n_rows: int, max_keys: int = 0) -> Batch:
    """New rows of a batch: sequence b has rows start[b] .. start[b+1] - 1 of the
    row tensors (n_rows of them), the first at position pos[b]; int32 device
    tensors [n_seqs + 1] and [n_seqs].  max_keys: about the most keys a sequence has
    (0: the cache's capacity); only the split of the work depends on it."""
    dev = _gpu(start, "start")
    n = start.shape[0] - 1 if start.dim() == 1 else 0
    if n < 1:
        _refuse("start: must be [n_seqs + 1]")
    b = Batch(_dense(start, torch.int32, (n + 1,), "start", dev),
              _dense(pos, torch.int32, (n,), "pos", dev), n, n_rows, max_keys)
    b.keep, b.device = (start, pos), dev
    return b


def _same(kv, b):
    if kv.device != b.device and kv.device is not None:   # None: a struct filled by hand
        _refuse("the batch and the cache must be on one device")
    if kv.n_seqs != b.n_seqs:
        _refuse("page_table and batch must have the same number of sequences")
    return b.device


def kv_append(k, v, kv: KVCache, layer: int, batch: Batch, stream=None):
    """Copy the batch's new rows (bf16 [n_rows, n_heads_kv, head_dim], rows may
    be strided) into one layer of a paged_kv cache."""
    _append_rows(_kv_append, k, v, kv, layer, batch, stream)


def kv8_append(k, v, kv: KV8Cache, layer: int, batch: Batch, stream=None):
    """Quantise the batch's new rows into one layer of a paged_kv8 cache."""
    _append_rows(_kv8_append, k, v, kv, layer, batch, stream)


def _append_rows(fn, k, v, kv, layer, batch, stream):
    dev = _same(kv, batch)
    n, h, d = batch.n_rows, kv.n_heads_kv, kv.head_dim
    ldk, ldv = _rows(k, n, h, d, "k", dev), _rows(v, n, h, d, "v", dev)
    _run(fn, dev, stream, k.data_ptr(), ldk, v.data_ptr(), ldv, kv, layer, batch)


def rope(head_dim: int, theta: float = 10000.0, freqs=None) -> Rope:
    """The rotation of position embeddings: pair (i, i + head_dim / 2) of a head turns by
    freqs[i] radians per position (a sequence of head_dim / 2 numbers; without it
    theta ** (-2 i / head_dim))."""
    r = Rope()
    f = None
    if freqs is not None:
        f = [float(x) for x in freqs]
        if 2 * len(f) != head_dim:
            _refuse("freqs: must be head_dim / 2 numbers")
        f = (C.c_double * len(f))(*f)
    _check(_rope_init(head_dim, theta, f, C.byref(r)))
    return r


def kv_append_rope(q, k, v, kv, layer: int, batch: Batch, rope: Rope, at=None, q_out=None,
                   stream=None):
    """Turn the batch's new rows q, k (bf16 [n_rows, heads, head_dim], rows may be strided)
    to their positions and write k and v into one layer of a paged_kv or paged_kv8 cache
    -> q turned.  at: int32 [n_rows], positions to turn to (None: where the rows stand;
    nodes of a tree: by their depth).  q_out may be q; rows of no sequence are left as
    they are in it, zero without.  q None: nothing but the cache is written."""
    dev = _same(kv, batch)
    n, h, d = batch.n_rows, kv.n_heads_kv, kv.head_dim
    ldk, ldv = _rows(k, n, h, d, "k", dev), _rows(v, n, h, d, "v", dev)
    qa = oa = None
    hq = ldq = ldo = 0
    if q is not None:
        if q.dim() != 3:
            _refuse("q: must be [n_rows, n_heads_q, head_dim]")
        hq = q.shape[1]
        ldq = _rows(q, n, hq, d, "q", dev)
        if q_out is None:
            q_out = _new((n, hq, d), torch.bfloat16, dev, stream, True)
        ldo = _rows(q_out, n, hq, d, "q_out", dev)
        qa, oa = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        _refuse("q_out without q")
    _run(_kv8_append_rope if type(kv) is KV8Cache else _kv_append_rope, dev, stream, qa, ldq, hq,
         k.data_ptr(), ldk, v.data_ptr(), ldv, kv, layer, batch, rope,
         None if at is None else _dense(at, torch.int32, (n,), "at", dev), oa, ldo)
    return q_out


def kv_move(kv, to, src, count, stream=None):
    """Move rows of a paged_kv or paged_kv8 cache within their sequences, in all layers: the
    row at position src[b, i] goes to position to[b] + i, for i < count[b] (int32 [n_seqs,
    n_max], [n_seqs], [n_seqs]; n_max <= 128).  All are read before any is written."""
    dev = _gpu(src, "src")
    if kv.device != dev and kv.device is not None:
        _refuse("src and the cache must be on one device")
    if src.dim() != 2 or src.shape[0] != kv.n_seqs:
        _refuse("src: must be [n_seqs, n_max]")
    n, most = src.shape
    _run(_kv8_move if type(kv) is KV8Cache else _kv_move, dev, stream, kv, n,
         _dense(to, torch.int32, (n,), "to", dev), _dense(src, torch.int32, (n, most), "src", dev),
         most, _dense(count, torch.int32, (n,), "count", dev))


def kv8_read(kv: KV8Cache, layer: int, batch: Batch, out=None, stream=None):
    """The values at the batch's positions -> (k, v) bf16 [n_rows, n_heads_kv,
    head_dim].  Rows of no sequence are left as they are in `out`, zero without."""
    dev = _same(kv, batch)
    shape = (batch.n_rows, kv.n_heads_kv, kv.head_dim)
    if out is None:
        out = (_new(shape, torch.bfloat16, dev, stream, True),
               _new(shape, torch.bfloat16, dev, stream, True))
    k, v = out
    _run(_kv8_read, dev, stream, kv, layer, batch,
         _dense(k, torch.bfloat16, shape, "out[0]", dev),
         _dense(v, torch.bfloat16, shape, "out[1]", dev))
    return k, v


def chunk_attn_workspace(n_heads_q: int, n_heads_kv: int, head_dim: int, n_seqs: int,
                         n_rows: int) -> int:
    """Bytes of workspace that a chunk_attn call of these sizes on the current device may
    need."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    return _workspace_bytes(dev, n_heads_q, n_heads_kv, head_dim, n_seqs, n_rows)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(device: int, *sizes) -> int:
    if device >= 0 and torch.cuda.current_device() != device:
        with torch.cuda.device(device):
            return _workspace_bytes(device, *sizes)
    n = _i64()
    _check(_chunk_attn_workspace(*sizes, C.byref(n)))
    return n.value


def chunk_attn(q, kv, layer: int, batch: Batch, scale=None, out=None, workspace=None,
               stream=None):
    """Causal attention of the batch's new rows (bf16 [n_rows, n_heads_q,
    head_dim], rows may be strided) over a paged_kv or paged_kv8 cache that holds
    their own keys already -> bf16 [n_rows, n_heads_q, head_dim].  Rows of no
    sequence are left as they are in `out`, zero without.  workspace: a uint8
    tensor of chunk_attn_workspace bytes; allocated by torch if not given."""
    return _attend(_chunk_attn8 if type(kv) is KV8Cache else _chunk_attn, q, kv, layer, batch,
                   _same(kv, batch), (), scale, out, workspace, stream)


def _attend(fn, q, kv, layer, batch, dev, extra, scale, out, workspace, stream):
    if q.dim() != 3:
        _refuse("q: must be [n_rows, n_heads_q, head_dim]")
    n, hq, d = batch.n_rows, q.shape[1], kv.head_dim
    ldq = _rows(q, n, hq, d, "q", dev)
    if out is None:
        out = _new((n, hq, d), torch.bfloat16, dev, stream, True)
    at = _dense(out, torch.bfloat16, (n, hq, d), "out", dev)
    args = (q.data_ptr(), ldq, hq, kv, layer, batch, *extra, d ** -0.5 if scale is None else scale, at)
    if workspace is None:
        size = _workspace_bytes(dev.index, hq, kv.n_heads_kv, d, batch.n_seqs, n)
        _run_scratch(fn, dev, stream, size, *args)
    else:
        ws = _dense(workspace, torch.uint8, workspace.shape, "workspace", dev)
        _run(fn, dev, stream, *args, ws or None, workspace.numel())
    return out


def chunk_tree_attn(q, kv, layer: int, batch: Batch, base, mask, scale=None, out=None,
                    workspace=None, stream=None):
    """chunk_attn for nodes of trees: row i of sequence b reads the keys up to its own
    position that are committed (before base[b], int32 [n_seqs]) or whose slot, counted from
    base[b], is set in its mask (int32 [n_rows, words], bit s % 32 of word s / 32: its path,
    itself included)."""
    dev = _same(kv, batch)
    if mask.dim() != 2:
        _refuse("mask: must be [n_rows, words]")
    words = mask.shape[1]
    extra = (_dense(base, torch.int32, (batch.n_seqs,), "base", dev),
             _dense(mask, torch.int32, (batch.n_rows, words), "mask", dev), words)
    return _attend(_chunk_tree_attn8 if type(kv) is KV8Cache else _chunk_tree_attn, q, kv, layer,
                   batch, dev, extra, scale, out, workspace, stream)


def beam_workspace(n_seqs: int, n_beams: int, vocab: int) -> int:
    """Bytes of workspace that a beam_select call of these sizes needs."""
    n = _i64()
    _check(_beam_workspace(n_seqs, n_beams, vocab, C.byref(n)))
    return n.value


def beam_select(logits, score, n_best: int, temperature: float = 1.0, state=None, slot: int = -1,
                out=None, workspace=None, stream=None):
    """The best continuations of each sequence's beams by one token: logits fp32 [n_seqs,
    n_beams, V], score fp32 [n_seqs, n_beams] (-inf: no beam) -> (token, parent int32, score
    fp32 [n_seqs, n_best]) in falling order of score + log_softmax(logits / temperature); -1,
    -1, -inf where there are fewer.  With state (int32 [n_seqs, n_beams, words]) also the
    parents' states [n_seqs, n_best, words]; slot >= 0 sets bit slot + r in the r-th of them
    (chunk_tree_attn's masks of a tree's next level)."""
    dev = _gpu(logits, "logits")
    if logits.dim() != 3:
        _refuse("logits: must be [n_seqs, n_beams, V]")
    b, n, v = logits.shape
    words = 0
    if state is not None:
        if state.dim() != 3:
            _refuse("state: must be [n_seqs, n_beams, words]")
        words = state.shape[2]
    shapes = ((b, n_best),) * 3 + ((b, n_best, words),) * (state is not None)
    if out is None:
        if n_best < 1:
            _refuse("n_best must be at least 1")
        out = tuple(_new(s, t, dev, stream, False) for s, t in zip(shapes, _BEAM_TYPES))
        at = [x.data_ptr() for x in out]
    else:
        if len(out) != len(shapes):
            _refuse("out: must be token, parent, score and, with state, the new states")
        at = [_dense(x, t, s, f"out[{i}]", dev) for i, (x, s, t) in enumerate(zip(out, shapes, _BEAM_TYPES))]
    args = (_dense(logits, torch.float32, (b, n, v), "logits", dev),
            _dense(score, torch.float32, (b, n), "score", dev), b, n, v, temperature, n_best,
            None if state is None else _dense(state, torch.int32, (b, n, words), "state", dev), words,
            slot, at[0], at[1], at[2], at[3] if state is not None else None)
    if workspace is None:
        _run_scratch(_beam_select, dev, stream, _beam_bytes(b, n, v), *args)
    else:
        ws = _dense(workspace, torch.uint8, workspace.shape, "workspace", dev)
        _run(_beam_select, dev, stream, *args, ws or None, workspace.numel())
    return tuple(out)


_BEAM_TYPES = (torch.int32, torch.int32, torch.float32, torch.int32)
_beam_bytes = functools.lru_cache(maxsize=4096)(beam_workspace)


def probs(logits, temperature: float = 1.0, out=None, stream=None):
    """softmax(logits / temperature) of fp32 [rows, V]; `out` may be the logits."""
    dev = _gpu(logits, "logits")
    if logits.dim() != 2:
        _refuse("logits: must be [rows, V]")
    shape = logits.shape
    z = _dense(logits, torch.float32, shape, "logits", dev)
    if out is None:
        out = _new(shape, torch.float32, dev, stream, False)
    _run(_probs, dev, stream, z, shape[0], shape[1], temperature,
         _dense(out, torch.float32, shape, "out", dev))
    return out


def verify_sample(p, q, draft, u, out=None, stream=None):
    """Verify drafted tokens against probabilities from given random numbers:
    p fp32 [n_seqs, n_draft + 1, V] the target's, q fp32 [n_seqs, n_draft, V] the
    draft's (None: its tokens were certain), draft int32 [n_seqs, n_draft] (the first
    entry outside [0, V) ends a sequence's draft), u fp32 [n_seqs, n_draft + 1] in
    [0, 1) -> (tokens int32 [n_seqs, n_draft + 1]: the accepted ones, the sampled one,
    then -1; n_accepted int32 [n_seqs]).  draft None: plain sampling from p."""
    dev = _gpu(p, "p")
    if p.dim() != 3 or p.shape[1] < 1:
        _refuse("p: must be [n_seqs, n_draft + 1, V]")
    b, n, v = p.shape
    n -= 1
    if draft is None and n > 0:
        _refuse("draft: must be [n_seqs, n_draft]")
    pa = _dense(p, torch.float32, p.shape, "p", dev)
    qa = None if q is None else _dense(q, torch.float32, (b, n, v), "q", dev)
    da = None if draft is None else _dense(draft, torch.int32, (b, n), "draft", dev)
    ua = _dense(u, torch.float32, (b, n + 1), "u", dev)
    if out is None:
        out = (_new((b, n + 1), torch.int32, dev, stream, False),
               _new((b,), torch.int32, dev, stream, False))
    tokens, n_accepted = out
    _run(_verify_sample, dev, stream, pa, qa if n else None, da if n else None, ua, b, n, v,
         _dense(tokens, torch.int32, (b, n + 1), "out[0]", dev),
         _dense(n_accepted, torch.int32, (b,), "out[1]", dev))
    return tokens, n_accepted


# -------------------------------------------------------------------- model --
class Model:
    """A decoder for SubSpec decoding: resident layers on the device, offloaded
    layers as pinned host originals (streamed for the target) plus device int4
    substitutes (packed here with the library's w4_pack) for the draft."""

    def __init__(self, cfg, weights: dict, max_seq: int, max_depth: int, max_width: int,
                 max_prompt: int | None = None, staging_layers: int = 0, device="cuda",
                 embed_on_host: bool = False, bits=4, hqq_iters: int = 0):
        """bits: code bits of the substitutes (2, 3 or 4), or one entry per
        layer (entries of resident layers are ignored) for mixed precision.
        hqq_iters > 0 packs them with the HQQ-optimised zero point."""
        self.cfg = cfg
        self.keep = []          # tensors the library points into
        self.w4 = {}            # (layer, name) -> (q, scale, zero) device substitutes
        dev = torch.device(device)

        def dev_t(t):
            t = t.to(dev, non_blocking=False).contiguous()
            self.keep.append(t)
            return t

        # the offloaded originals live in one pinned host arena (one large
        # page-locked allocation), each matrix 256-byte aligned inside it
        names = ("wq", "wk", "wv", "wo", "wg", "wu", "wd")
        off_mats = [(i, n) for i in range(cfg.n_resident, cfg.n_layers) for n in names]
        sizes = [weights["layers"][i][n].numel() * 2 for i, n in off_mats]
        total = sum((b + 255) // 256 * 256 for b in sizes)
        arena = torch.empty(max(total, 256), dtype=torch.uint8, pin_memory=True)
        self.keep.append(arena)
        host_of, pos = {}, 0
        for (i, n), b in zip(off_mats, sizes):
            w = weights["layers"][i][n]
            view = arena[pos:pos + b].view(torch.bfloat16).view(w.shape)
            view.copy_(w)
            host_of[(i, n)] = view
            pos += (b + 255) // 256 * 256

        layers = (LayerDesc * cfg.n_layers)()
        for i, lw in enumerate(weights["layers"]):
            L = layers[i]
            L.attn_norm = dev_t(lw["attn_norm"]).data_ptr()
            L.ffn_norm = dev_t(lw["ffn_norm"]).data_ptr()
            w4n = ("q4", "k4", "v4", "o4", "g4", "u4", "d4")
            for name, qn in zip(names, w4n):
                w = lw[name]
                if i < cfg.n_resident:
                    setattr(L, name, dev_t(w).data_ptr())
                else:
                    b = bits[i] if isinstance(bits, (list, tuple)) else bits
                    wd = w.to(dev).contiguous()
                    if hqq_iters > 0:
                        q, s, z = wq_pack_hqq(wd, b, hqq_iters)
                    else:
                        q, s, z = w4_pack(wd) if b == 4 else wq_pack(wd, b)
                    self.w4[(i, name)] = (q, s, z)
                    setattr(L, qn, W4(q.data_ptr(), s.data_ptr(), z.data_ptr(), b))
                    setattr(L, name, host_of[(i, name)].data_ptr())
                    del wd
        torch.cuda.synchronize(dev)
        d = ModelDesc()
        for f in ("n_layers", "hidden", "n_heads_q", "n_heads_kv", "head_dim", "ffn", "vocab",
                  "n_resident"):
            setattr(d, f, getattr(cfg, f))
        d.rope_theta = cfg.rope_theta
        d.rms_eps = cfg.rms_eps
        if embed_on_host:   # read in place from pinned host memory
            emb = weights["embed"].to("cpu").contiguous().pin_memory()
            self.keep.append(emb)
            d.embed = emb.data_ptr()
        else:
            d.embed = dev_t(weights["embed"]).data_ptr()
        d.lm_head = dev_t(weights["lm_head"]).data_ptr()
        d.final_norm = dev_t(weights["final_norm"]).data_ptr()
        d.layers = layers
        d.max_seq = max_seq
        d.max_depth = max_depth
        d.max_width = max_width
        d.staging_layers = staging_layers
        d.max_prompt = max_prompt if max_prompt is not None else max_seq
        self._layers = layers
        h = _vp()
        _check(_model_create(C.byref(d), C.byref(h)))
        self.handle = h
        self.device = torch.device("cuda", torch.cuda.current_device())   # of its pools

    def close(self):
        """Destroy the model and drop the tensors it pointed into (the pinned
        originals and the device substitutes)."""
        if getattr(self, "handle", None) and self.handle.value:
            _model_destroy(self.handle)
            self.handle = _vp()
        self.keep = []
        self.w4 = {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def device_bytes(self) -> int:
        b = _i64()
        _check(_model_memory(self.handle, C.byref(b)))
        return b.value

    def kv(self) -> KVCache:
        """The cache of the model's one sequence.  Keeps the model; not valid after close()."""
        kv = KVCache()
        _check(_model_kv(self.handle, C.byref(kv)))
        kv.keep, kv.device = (self,), self.device
        return kv

    def forward(self, which: int, tokens, slot0: int, n_prefix: int, depth=None, anc=None,
                logits=None, stream=None):
        n = tokens.shape[0]
        _check(_model_forward(self.handle, which, _p(tokens), n, slot0, _p(depth), _p(anc),
                              0 if anc is None else anc.shape[1], n_prefix, _p(logits),
                              _stream(stream)))
        return logits

    @staticmethod
    def decode_cfg(depth, width, draft_temp=0.2, mode=0, target_temp=1.0, seed=0,
                   use_graph=True, stop_logp=None, verify_reuse=False) -> DecodeCfg:
        """stop_logp: None (every level drafted) or a negative threshold for adaptive
        depth; verify_reuse: the verify starts from the draft's leading layers."""
        return DecodeCfg(depth, width, draft_temp, mode, target_temp, seed, int(use_graph),
                         0.0 if stop_logp is None else float(stop_logp), int(verify_reuse))

    def prefill(self, prompt, cfg: DecodeCfg, stream=None):
        self._prompt = prompt.to(torch.int32).contiguous()
        _check(_prefill(self.handle, C.c_void_p(self._prompt.data_ptr()), self._prompt.numel(),
                        C.byref(cfg), _stream(stream)))

    def decode_cycles(self, cfg: DecodeCfg, n_cycles: int, stream=None):
        _check(_decode_cycles(self.handle, C.byref(cfg), n_cycles, _stream(stream)))

    def decode_read(self, n: int = 0):
        """-> (emitted tokens int32 CPU tensor [min(n, emitted)], emitted, cycles)."""
        out = torch.zeros(max(n, 1), dtype=torch.int32)
        e, c = _i32(), _i64()
        _check(_decode_read(self.handle, C.c_void_p(out.data_ptr()), n, C.byref(e), C.byref(c)))
        return out[:min(n, e.value)], e.value, c.value

    def cycle_info(self, cfg: DecodeCfg):
        k, b = _i64(), _i64()
        _check(_cycle_info(self.handle, C.byref(cfg), C.byref(k), C.byref(b)))
        return k.value, b.value

    def generate(self, prompt, n_new: int, depth: int, width: int, draft_temp=0.2, mode=0,
                 target_temp=1.0, seed=0, use_graph=True, stop_logp=None, verify_reuse=False):
        """prompt: int32 CPU tensor -> (int32 CPU tensor [n_new], Stats)."""
        p = prompt.to(torch.int32).contiguous()
        out = torch.zeros(n_new, dtype=torch.int32)
        cfg = self.decode_cfg(depth, width, draft_temp, mode, target_temp, seed, use_graph,
                              stop_logp, verify_reuse)
        st = Stats()
        _check(_generate(self.handle, C.c_void_p(p.data_ptr()), p.numel(), n_new, C.byref(cfg),
                         C.c_void_p(out.data_ptr()), C.byref(st)))
        return out, st
