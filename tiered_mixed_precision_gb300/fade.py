"""ctypes binding of libfade (argument marshalling only; every step runs in the CUDA library).

The functions keep the C names (``fade_quantize_pack``, ``fade_decode_attention``, ...).
Tensors are torch tensors on a CUDA device; their data pointers and the current CUDA stream
are passed to the C entry points. A missing library raises ``ImportError``: there is no CPU
fallback.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# FADE_LIBRARY=debug loads the FADE_DEBUG=1 build (build.build(debug=True)) instead
LIB_PATH = os.path.join(_PKG, "_build_debug" if os.environ.get("FADE_LIBRARY") == "debug"
                        else "_build", "libfade.so")

FADE_OK, FADE_ERR_INVALID_ARGUMENT, FADE_ERR_UNSUPPORTED, FADE_ERR_CAPACITY, FADE_ERR_CUDA = range(5)
ROPE_KINDS = {"none": 0, "default": 1, "llama3": 2, "linear": 3, "ntk": 4, "yarn": 5,
              "dynamic": 6}
POLICIES = {"none": 0, "h2o": 1, "ema": 2, "position": 3}
V_CODECS = {"int": 0, "pq": 1}
PQ_SUB, PQ_CENTROIDS, PQ_MAX_CALIB = 4, 256, 8192


def pq_train_ws_bytes(dim: int) -> int:
    """FADE_PQ_TRAIN_WS_BYTES(dim)."""
    return dim * 2304 + 1024
META_FIELDS = 8
META = {"n_sink": 0, "n_mid": 1, "n_recent": 2, "head": 3, "cur": 4, "n_ev": 5, "sync": 6}
MAX_BATCH = 256
STATUS_WORDS = 4
ATTN_TILE_TOKENS = 256   # FADE_ATTN_TILE_TOKENS
TREE_MAX_NODES = 64      # FADE_TREE_MAX_NODES


class FadeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libfade status {status}: {message}")
        self.status = status


c_i32, c_i64, c_f32, c_f64, c_sz, c_vp = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                                          ctypes.c_double, ctypes.c_size_t, ctypes.c_void_p)


class RopeT(ctypes.Structure):
    _fields_ = [("kind", c_i32), ("original_max_position", c_i32), ("base", c_f64),
                ("factor", c_f64), ("low_freq_factor", c_f64), ("high_freq_factor", c_f64),
                ("rotary_dim", c_i32)]


class ConfigT(ctypes.Structure):
    _fields_ = [("batch", c_i32), ("num_q_heads", c_i32), ("num_kv_heads", c_i32),
                ("head_dim", c_i32), ("n_sink", c_i32), ("recent_window", c_i32),
                ("int4_budget", c_i32), ("middle_k_bits", c_i32), ("middle_v_bits", c_i32),
                ("mid_capacity", c_i32), ("policy", c_i32), ("ema_decay", c_f32),
                ("shared_rows", c_i32), ("v_codec", c_i32), ("rope", RopeT)]


class LayerT(ctypes.Structure):
    _fields_ = [("sink_k", c_vp), ("sink_v", c_vp), ("recent_k", c_vp), ("recent_v", c_vp),
                ("mid_k_codes", c_vp * 2), ("mid_k_scales", c_vp * 2),
                ("mid_v_codes", c_vp * 2), ("mid_v_scales", c_vp * 2),
                ("sink_scores", c_vp), ("mid_scores", c_vp * 2), ("recent_scores", c_vp),
                ("meta", c_vp), ("victims", c_vp), ("chunk_base", c_vp),
                ("victim_words", c_i32), ("chunk_slots", c_i32), ("status", c_vp),
                ("h_n_sink", c_vp), ("h_n_mid", c_vp), ("h_n_recent", c_vp),
                ("pq_codebook", c_vp)]


class HeadsT(ctypes.Structure):
    _fields_ = [("x", c_vp), ("row_stride", c_i64), ("token_stride", c_i64),
                ("head_stride", c_i64)]


class LogitsT(ctypes.Structure):
    _fields_ = [("x", c_vp), ("row_stride", c_i64), ("node_stride", c_i64)]


class LayoutT(ctypes.Structure):
    _fields_ = [(n, c_sz) for n in (
        "sink_k", "sink_v", "recent_k", "recent_v", "mid_k_codes", "mid_k_scales",
        "mid_v_codes", "mid_v_scales", "sink_scores", "mid_scores", "recent_scores", "meta",
        "victims", "chunk_base", "status", "logits_ws")] + [("mid_stride", c_i32)] + [
        (n, c_sz) for n in ("ml_ws", "attn_ws")] + [
        ("victim_words", c_i32), ("chunk_slots", c_i32), ("max_prompt", c_i32),
        ("max_splits", c_i32), ("prefill_mass_ws", c_sz)]


_lib = None


def lib():
    """The loaded libfade (ImportError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libfade is not built ({LIB_PATH} missing): run "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        S = ctypes.POINTER
        sig = {
            "fade_layout": (c_i32, [S(ConfigT), c_i32, S(LayoutT)]),
            "fade_rope_table_init": (c_i32, [S(ConfigT), c_vp, c_i32, c_vp]),
            "fade_rope_apply": (c_i32, [S(ConfigT), c_vp, c_i32, c_vp, c_vp, c_i64, c_i32,
                                        c_vp, c_i32, c_vp]),
            "fade_quantize_pack": (c_i32, [c_vp, c_i64, c_i32, c_i32, c_vp, c_vp, c_vp]),
            "fade_dequantize": (c_i32, [c_vp, c_vp, c_i64, c_i32, c_i32, c_vp, c_vp]),
            "fade_cache_reset": (c_i32, [S(ConfigT), S(LayerT), c_vp]),
            "fade_cache_prefill": (c_i32, [S(ConfigT), S(LayerT), c_vp, c_vp, c_i32, c_vp,
                                           c_vp, c_vp, c_i32, c_vp]),
            "fade_prefill_mass": (c_i32, [S(ConfigT), c_vp, c_vp, c_i32, c_vp, c_vp, c_vp,
                                          c_sz, c_vp]),
            "fade_cache_demote": (c_i32, [S(ConfigT), S(LayerT), c_vp]),
            "fade_evict_rerope": (c_i32, [S(ConfigT), S(LayerT), c_vp, c_i32, c_vp]),
            "fade_cache_append": (c_i32, [S(ConfigT), S(LayerT), c_vp, c_vp, c_vp]),
            "fade_rope_append": (c_i32, [S(ConfigT), S(LayerT), c_vp, c_i32, c_vp, c_vp, c_vp,
                                         c_vp, c_vp, c_i32, c_vp]),
            "fade_decode_attention": (c_i32, [S(ConfigT), S(LayerT), c_vp, c_vp, c_vp, c_vp,
                                              c_vp, c_sz, c_vp]),
            "fade_h2o_accumulate": (c_i32, [S(ConfigT), S(LayerT), c_vp, c_vp, c_vp]),
            "fade_next_position": (c_i32, [S(ConfigT), S(LayerT), c_i32]),
            "fade_compressed_bytes": (ctypes.c_uint64, [S(ConfigT), S(LayerT)]),
            "fade_cache_advance_host": (c_i32, [S(ConfigT), S(LayerT)]),
            "fade_cache_advance_host_layers": (c_i32, [S(ConfigT), c_vp, c_i32]),
            "fade_pq_encode": (c_i32, [c_vp, c_vp, c_i64, c_i32, c_vp, c_vp]),
            "fade_pq_decode": (c_i32, [c_vp, c_vp, c_i64, c_i32, c_vp, c_vp]),
            "fade_pq_train": (c_i32, [c_vp, c_i64, c_i32, c_vp, c_i32, c_vp, c_vp, c_sz, c_vp]),
            "fade_check_status": (c_i32, [S(LayerT), c_vp]),
            "fade_tier_counts": (c_i32, [S(ConfigT), S(LayerT), c_vp]),
            "fade_attention_tiled": (c_i32, [S(ConfigT)]),
            "fade_measure_fp32_rate": (c_i32, [c_i32, c_i32, c_vp, ctypes.POINTER(c_f64), c_vp]),
            "fade_selftest_bounded_wait": (c_i32, [c_vp, c_i32, c_i64, c_vp]),
            "fade_tree_layout": (c_i32, [S(ConfigT), c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
            "fade_qk_norm_rope": (c_i32, [S(ConfigT), c_vp, c_i32, S(HeadsT), S(HeadsT), c_vp,
                                          S(HeadsT), S(HeadsT), c_vp, c_f32, c_vp, c_i64, c_i32,
                                          c_vp]),
            "fade_tree_ws_bytes": (c_sz, [S(ConfigT), c_i32]),
            "fade_tree_attention": (c_i32, [S(ConfigT), S(LayerT), c_i32, c_vp, S(HeadsT),
                                            S(HeadsT), c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
            "fade_tree_commit": (c_i32, [S(ConfigT), S(LayerT), c_i32, c_vp, c_vp, S(HeadsT),
                                         S(HeadsT), c_vp, c_vp, c_vp, c_sz, c_vp]),
            "fade_tree_verify": (c_i32, [S(ConfigT), c_i32, c_i32, c_i32, c_vp, c_vp, c_vp,
                                         S(LogitsT), S(LogitsT), S(LogitsT), S(LogitsT), c_vp, c_vp,
                                         c_vp, c_vp, c_vp, c_vp, c_vp]),
            "fade_prompt_ws_bytes": (c_sz, [S(ConfigT), c_i32, c_i32]),
            "fade_prompt_attention": (c_i32, [S(ConfigT), S(HeadsT), S(HeadsT), S(HeadsT), c_i32,
                                              c_i32, c_vp, c_vp, c_i32, c_i32, S(HeadsT), c_vp,
                                              c_vp, c_vp, c_sz, c_vp]),
            "fade_prompt_mass": (c_i32, [S(ConfigT), S(HeadsT), S(HeadsT), c_i32, c_i32, c_vp, c_vp,
                                         c_i32, c_i32, c_vp, c_i32, c_vp, c_vp, c_vp, c_sz, c_vp]),
            "fade_last_error": (ctypes.c_char_p, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def fade_last_error() -> str:
    return lib().fade_last_error().decode()


def _check(status: int):
    if status != FADE_OK:
        raise FadeError(status, fade_last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = None


def _stream(stream):
    """The handle of ``stream``, or of the current CUDA stream (the raw-handle query when
    torch has it: it skips building a Stream object on every call)."""
    global _raw_stream
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    import torch

    if _raw_stream is None:
        fn = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = ((lambda: fn(torch.cuda.current_device())) if fn is not None
                       else (lambda: torch.cuda.current_stream().cuda_stream))
    return ctypes.c_void_p(_raw_stream())


# --------------------------------------------------------------------------- config
@dataclass
class Config:
    """One layer's cache configuration (the FadeConfig fields plus shapes)."""
    batch: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    n_sink: int = 4
    recent_window: int = 64
    int4_budget: int = -1
    middle_k_bits: int = 4
    middle_v_bits: int = 2
    mid_capacity: int = 0
    policy: str = "none"
    ema_decay: float = 0.9
    rope_kind: str = "default"
    rope_base: float = 10000.0
    rope_factor: float = 1.0
    rope_low_freq_factor: float = 1.0
    rope_high_freq_factor: float = 4.0
    rope_original_max_position: int = 8192
    rope_rotary_dim: int = 0   # proportional RoPE: rotated channels (0 = every channel)
    shared_rows: bool = False  # the rows share their tier decisions (row-summed scores)
    v_codec: str = "int"       # "pq": product-quantised middle V (needs middle_v_bits = 2)
    _c: ConfigT = field(default=None, init=False, repr=False, compare=False)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name != "_c":   # any change of a field invalidates the cached C struct
            object.__setattr__(self, "_c", None)

    def c(self) -> ConfigT:
        """The C struct (built once per set of field values: every entry point takes it)."""
        if self._c is None:
            r = RopeT(ROPE_KINDS[self.rope_kind], self.rope_original_max_position,
                      self.rope_base, self.rope_factor, self.rope_low_freq_factor,
                      self.rope_high_freq_factor, self.rope_rotary_dim)
            object.__setattr__(self, "_c", ConfigT(
                self.batch, self.num_q_heads, self.num_kv_heads, self.head_dim, self.n_sink,
                self.recent_window, self.int4_budget, self.middle_k_bits, self.middle_v_bits,
                self.mid_capacity, POLICIES[self.policy], self.ema_decay,
                int(self.shared_rows), V_CODECS[self.v_codec], r))
        return self._c

    @property
    def group(self):
        return self.num_q_heads // self.num_kv_heads

    @property
    def evicts(self):
        return self.policy != "none" and self.int4_budget >= 0

    @classmethod
    def from_workload(cls, wl, mid_capacity=None, batch=None) -> "Config":
        evicts = wl.policy != "none" and wl.int4_budget >= 0
        if mid_capacity is None:
            if evicts:
                mid_capacity = wl.int4_budget + 1
            else:
                longest = wl.ragged[1] if wl.ragged else wl.prompt_len
                mid_capacity = max(1, longest + wl.steps - wl.n_sink - wl.recent_window)
        r = wl.rope
        return cls(batch or wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.n_sink,
                   wl.recent_window, wl.int4_budget, wl.middle_k_bits, wl.middle_v_bits,
                   mid_capacity, wl.policy, wl.ema_decay, r.kind, r.base, r.factor,
                   r.low_freq_factor, r.high_freq_factor, r.original_max_position,
                   getattr(r, "rotary_dim", 0))


def preset(name: str, batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
           **kw) -> Config:
    """The pages' presets as configurations: "safe" (no eviction, INT4 K and V), "balanced"
    (H2O, budget 400, INT4 K / INT2 V), "aggressive" (position eviction, INT4 K / INT2 V,
    budget 4096 unless given)."""
    base = dict(batch=batch, num_q_heads=num_q_heads, num_kv_heads=num_kv_heads,
                head_dim=head_dim, n_sink=4, recent_window=64)
    if name == "safe":
        base.update(policy="none", int4_budget=-1, middle_k_bits=4, middle_v_bits=4)
    elif name == "balanced":
        base.update(policy="h2o", int4_budget=400, middle_k_bits=4, middle_v_bits=2)
    elif name == "aggressive":
        base.update(policy="position", int4_budget=4096, middle_k_bits=4, middle_v_bits=2)
    else:
        raise ValueError(f"unknown preset {name!r}")
    base.update(kw)
    if "mid_capacity" not in kw:
        base["mid_capacity"] = base["int4_budget"] + 1 if base["int4_budget"] >= 0 else 8192
    return Config(**base)


def fade_layout(cfg: Config, max_prompt: int) -> LayoutT:
    out = LayoutT()
    _check(lib().fade_layout(ctypes.byref(cfg.c()), max_prompt, ctypes.byref(out)))
    return out


# --------------------------------------------------------------------------- layer buffers
class TieredLayer:
    """Device buffers of one layer (torch-allocated) plus the host mirror of tier counts."""

    def __init__(self, cfg: Config, max_prompt: int, device="cuda"):
        import torch

        self.cfg = cfg
        self.layout = lay = fade_layout(cfg, max_prompt)
        B, H, d = cfg.batch, cfg.num_kv_heads, cfg.head_dim
        S, W, C = cfg.n_sink, cfg.recent_window, lay.mid_stride
        dev = torch.device(device)
        u8, f16, f32, i32 = torch.uint8, torch.float16, torch.float32, torch.int32
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)
        self.sink_k = z((B, H, S, d), f16)
        self.sink_v = z((B, H, S, d), f16)
        self.recent_k = z((B, H, W, d), f16)
        self.recent_v = z((B, H, W, d), f16)
        self.mid_k_codes = [z((B, H, C, d * cfg.middle_k_bits // 8), u8) for _ in range(2)]
        self.mid_k_scales = [z((B, H, C, d // 32), f16) for _ in range(2)]
        self.mid_v_codes = [z((B, H, C, d * cfg.middle_v_bits // 8), u8) for _ in range(2)]
        self.mid_v_scales = [z((B, H, C, d // 32), f16) for _ in range(2)]
        self.sink_scores = z((B, H, max(S, 0)), f32)
        self.mid_scores = [z((B, H, C), f32) for _ in range(2)]
        self.recent_scores = z((B, H, W), f32)
        self.meta = z((B, H, META_FIELDS), i32)
        self.victims = z((B, H, lay.victim_words), torch.int32)
        self.chunk_base = z((B, H, lay.chunk_slots), i32)
        self.status = z((STATUS_WORDS,), i32)
        self.h_n_sink = np.zeros(B, np.int32)
        self.h_n_mid = np.zeros(B, np.int32)
        self.h_n_recent = np.zeros(B, np.int32)
        # the layer's PQ codebook (product-quantised V only): fp16 [d/4][256][4]
        self.pq_codebook = z((d // PQ_SUB, PQ_CENTROIDS, PQ_SUB), f16) if cfg.v_codec == "pq" else None
        self.pq_codebook_set = False   # PQ: encoding needs a codebook installed first
        p = lambda t: t.data_ptr()
        self.c = LayerT(
            p(self.sink_k), p(self.sink_v), p(self.recent_k), p(self.recent_v),
            (c_vp * 2)(*map(p, self.mid_k_codes)), (c_vp * 2)(*map(p, self.mid_k_scales)),
            (c_vp * 2)(*map(p, self.mid_v_codes)), (c_vp * 2)(*map(p, self.mid_v_scales)),
            p(self.sink_scores), (c_vp * 2)(*map(p, self.mid_scores)), p(self.recent_scores),
            p(self.meta), p(self.victims), p(self.chunk_base), lay.victim_words,
            lay.chunk_slots, p(self.status), self.h_n_sink.ctypes.data, self.h_n_mid.ctypes.data,
            self.h_n_recent.ctypes.data,
            None if self.pq_codebook is None else p(self.pq_codebook))

    def set_pq_codebook(self, codebook):
        """Copy a codebook (fp16 [d/4][256][4], e.g. from fade_pq_train) into the layer."""
        if self.pq_codebook is None:
            raise ValueError("the layer does not use product-quantised V")
        self.pq_codebook.copy_(codebook)
        self.pq_codebook_set = True

    def workspaces(self):
        """(logits_ws, ml_ws, attn_ws) tensors sized by the layout."""
        import torch

        dev = self.meta.device
        lay = self.layout
        return (torch.empty(lay.logits_ws // 4, dtype=torch.float32, device=dev),
                torch.empty(lay.ml_ws // 4, dtype=torch.float32, device=dev),
                torch.empty(lay.attn_ws, dtype=torch.uint8, device=dev))


# --------------------------------------------------------------------------- entry points
def fade_rope_table_init(cfg: Config, table, max_pos: int, stream=None):
    _check(lib().fade_rope_table_init(ctypes.byref(cfg.c()), _ptr(table), max_pos, _stream(stream)))


def fade_rope_apply(cfg: Config, table, max_pos, x, y, n_groups, group_len, pos_start=None,
                    pos_step=1, stream=None):
    _check(lib().fade_rope_apply(ctypes.byref(cfg.c()), _ptr(table), max_pos, _ptr(x), _ptr(y),
                                 n_groups, group_len, _ptr(pos_start), pos_step, _stream(stream)))


def fade_quantize_pack(x, n_vec, dim, bits, codes, scales, stream=None):
    _check(lib().fade_quantize_pack(_ptr(x), n_vec, dim, bits, _ptr(codes), _ptr(scales),
                                    _stream(stream)))


def fade_dequantize(codes, scales, n_vec, dim, bits, out, stream=None):
    _check(lib().fade_dequantize(_ptr(codes), _ptr(scales), n_vec, dim, bits, _ptr(out),
                                 _stream(stream)))


def fade_cache_reset(layer: TieredLayer, stream=None):
    _check(lib().fade_cache_reset(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                  _stream(stream)))


def _require_codebook(layer: TieredLayer):
    if layer.pq_codebook is not None and not layer.pq_codebook_set:
        raise ValueError("product-quantised V: install the layer's codebook first "
                         "(set_pq_codebook, or FadeCache.train_pq_codebook)")


def fade_cache_prefill(layer: TieredLayer, k_rot, v, max_prompt, prompt_len, mass, table,
                       max_pos, stream=None):
    _require_codebook(layer)
    lens = np.ascontiguousarray(prompt_len, np.int32)
    _check(lib().fade_cache_prefill(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                    _ptr(k_rot), _ptr(v), max_prompt, lens.ctypes.data,
                                    _ptr(mass), _ptr(table), max_pos, _stream(stream)))


def fade_prefill_mass(cfg: Config, q_rot, k_rot, max_prompt, prompt_len, mass, ws=None,
                      stream=None):
    """ws: device workspace of at least layout(cfg, max_prompt).prefill_mass_ws bytes (made
    here when not given)."""
    lens = np.ascontiguousarray(prompt_len, np.int32)
    if ws is None:
        import torch

        ws = torch.empty(fade_layout(cfg, max_prompt).prefill_mass_ws, dtype=torch.uint8,
                         device=q_rot.device)
    nbytes = ws.numel() * ws.element_size()
    _check(lib().fade_prefill_mass(ctypes.byref(cfg.c()), _ptr(q_rot), _ptr(k_rot), max_prompt,
                                   lens.ctypes.data, _ptr(mass), _ptr(ws), nbytes,
                                   _stream(stream)))


def fade_cache_demote(layer: TieredLayer, stream=None):
    _require_codebook(layer)
    _check(lib().fade_cache_demote(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                   _stream(stream)))


def fade_evict_rerope(layer: TieredLayer, table, max_pos, stream=None):
    _check(lib().fade_evict_rerope(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                   _ptr(table), max_pos, _stream(stream)))


def fade_cache_append(layer: TieredLayer, k_rot, v, stream=None):
    _check(lib().fade_cache_append(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                   _ptr(k_rot), _ptr(v), _stream(stream)))


def fade_rope_append(layer: TieredLayer, table, max_pos, q_raw, k_raw, v, pos, q_rot,
                     demote=False, stream=None):
    """RoPE of q_raw into q_rot and of k_raw at pos[b] (device i32 [B]), and the append of the
    rotated key and v, in one launch (the same bits as fade_rope_apply twice and
    fade_cache_append); demote: fade_cache_demote first, in the same launch."""
    _check(lib().fade_rope_append(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                  _ptr(table), max_pos, _ptr(q_raw), _ptr(k_raw), _ptr(v),
                                  _ptr(pos), _ptr(q_rot), int(bool(demote)), _stream(stream)))


def fade_decode_attention(layer: TieredLayer, q_rot, out, logits_ws, ml_ws, ws, stream=None):
    _check(lib().fade_decode_attention(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                       _ptr(q_rot), _ptr(out), _ptr(logits_ws), _ptr(ml_ws),
                                       _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def fade_h2o_accumulate(layer: TieredLayer, logits_ws, ml_ws, stream=None):
    _check(lib().fade_h2o_accumulate(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                     _ptr(logits_ws), _ptr(ml_ws), _stream(stream)))


def fade_next_position(layer: TieredLayer, row: int) -> int:
    r = lib().fade_next_position(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c), row)
    if r < 0:
        raise FadeError(FADE_ERR_INVALID_ARGUMENT, fade_last_error())
    return r


def fade_cache_advance_host(layer: TieredLayer):
    _check(lib().fade_cache_advance_host(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c)))


def layer_pointer_array(layers):
    """A host array of the layers' C structs (for fade_cache_advance_host_layers); it stays
    valid while the layers live."""
    arr = (ctypes.POINTER(LayerT) * len(layers))(*[ctypes.pointer(L.c) for L in layers])
    return arr


def fade_cache_advance_host_layers(cfg: "Config", layer_array, n_layers: int):
    """fade_cache_advance_host for every layer of ``layer_array`` (``layer_pointer_array``)."""
    _check(lib().fade_cache_advance_host_layers(ctypes.byref(cfg.c()), layer_array, n_layers))


def fade_compressed_bytes(layer: TieredLayer) -> int:
    return int(lib().fade_compressed_bytes(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c)))


def fade_decode_attention_noalloc(layer: TieredLayer, q_rot, out, logits_ws, ml_ws, stream=None):
    """Decode attention with the split scratch inside the library (no workspace argument), for
    callers that cannot allocate device memory; see include/fade.h for its limits."""
    fn = lib().fade_decode_attention_noalloc
    fn.restype = c_i32
    fn.argtypes = [ctypes.POINTER(ConfigT), ctypes.POINTER(LayerT), c_vp, c_vp, c_vp, c_vp, c_vp]
    _check(fn(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c), _ptr(q_rot), _ptr(out),
              _ptr(logits_ws), _ptr(ml_ws), _stream(stream)))


def fade_pq_encode(codebook, x, n_vec, dim, codes, stream=None):
    _check(lib().fade_pq_encode(_ptr(codebook), _ptr(x), n_vec, dim, _ptr(codes),
                                _stream(stream)))


def fade_pq_decode(codebook, codes, n_vec, dim, out, stream=None):
    _check(lib().fade_pq_decode(_ptr(codebook), _ptr(codes), n_vec, dim, _ptr(out),
                                _stream(stream)))


def fade_pq_train(calib, n_vec, dim, init_idx, iters, codebook, ws, stream=None):
    """``init_idx``: 256 host row indices (any int sequence); ``ws``: a device tensor of at
    least pq_train_ws_bytes(dim) bytes."""
    idx = np.ascontiguousarray(init_idx, np.int32)
    if idx.shape != (PQ_CENTROIDS,):
        raise ValueError("init_idx must hold 256 indices")
    _check(lib().fade_pq_train(_ptr(calib), n_vec, dim, idx.ctypes.data, iters, _ptr(codebook),
                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def fade_check_status(layer: TieredLayer, stream=None):
    """Synchronise the stream and raise FadeError (status 5, FADE_ERR_TIMEOUT) if a kernel of
    the layer gave up a bounded wait since the last reset."""
    _check(lib().fade_check_status(ctypes.byref(layer.c), _stream(stream)))


def fade_selftest_bounded_wait(status, producer_arrives: bool, limit_cycles: int, stream=None):
    """Launch the bounded-wait self-test kernel (status: a device int32 tensor)."""
    _check(lib().fade_selftest_bounded_wait(_ptr(status), int(bool(producer_arrives)),
                                            int(limit_cycles), _stream(stream)))


def fade_measure_fp32_rate(blocks: int, iters: int, sink, stream=None) -> float:
    """Launch the fp32-rate measurement kernel; returns the fp32 operations it performs."""
    ops = c_f64(0.0)
    _check(lib().fade_measure_fp32_rate(int(blocks), int(iters), _ptr(sink), ctypes.byref(ops),
                                        _stream(stream)))
    return ops.value


_torch = None
_dtypes = {}         # by name, once torch is there
_available = False   # CUDA is (the query is not free)


def _device(stream):
    """The device the tensors of a call have to lie on: the current CUDA device, whose current
    stream the call is enqueued on; None if the caller passes its own stream (and answers for
    it)."""
    global _torch
    if _torch is None:
        import torch

        for name in ("float16", "bfloat16", "float32", "int32", "int64"):
            _dtypes[name] = getattr(torch, name)
        _torch = torch   # (last: another thread that sees it uses the types, too)
    if stream is not None:
        return None
    global _available
    _available = _available or _torch.cuda.is_available()
    return _torch.cuda.current_device() if _available else -2


def _tensor(device, name, t, dtype, shape, strided=False):
    """ValueError unless t (None: not given) has the dtype, shape and layout asked for (strided:
    only the last dimension has to be contiguous) and lies on the device."""
    if t is None:
        return
    if t.dtype is not _dtypes[dtype] or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, not "
                         f"{str(t.dtype).removeprefix('torch.')} {tuple(t.shape)}")
    if strided:
        if t.stride(-1) != 1 and t.numel():
            raise ValueError(f"{name} must be contiguous in its last dimension")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")


def _heads(t):
    """A [rows][tokens][heads][d] tensor as a fade_heads_t."""
    if t is None:
        return None
    rows, tokens, heads, _ = t.stride()
    return ctypes.byref(HeadsT(t.data_ptr(), rows, tokens, heads))


def _checked_heads(device, name, t, shape):
    """``_heads`` of a float16 tensor that ``_tensor`` would take as strided."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is _torch.float16 and t.shape == shape:
        rows, tokens, heads, one = t.stride()
        if one == 1 and (device is None or t.get_device() == device):
            return ctypes.byref(HeadsT(t.data_ptr(), rows, tokens, heads))
    _tensor(device, name, t, "float16", shape, True)
    return _heads(t)


def fade_tree_layout(cfg: Config, parents, n_nodes, base_pos, mask, pos, stream=None):
    """parents i32 [B][T], n_nodes i32 [B] or None, base_pos i32 [B] -> mask i64 [B][T] (the
    64 bits of FADE's u64 masks), pos i32 [B][T]."""
    B, T = parents.shape
    dev = _device(stream)
    _tensor(dev, "parents", parents, "int32", (cfg.batch, T))
    _tensor(dev, "n_nodes", n_nodes, "int32", (B,))
    _tensor(dev, "base_pos", base_pos, "int32", (B,))
    _tensor(dev, "mask", mask, "int64", (B, T))
    _tensor(dev, "pos", pos, "int32", (B, T))
    _check(lib().fade_tree_layout(ctypes.byref(cfg.c()), T, _ptr(parents), _ptr(n_nodes),
                                  _ptr(base_pos), _ptr(mask), _ptr(pos), _stream(stream)))


def fade_qk_norm_rope(cfg: Config, table, max_pos, q, k, q_weight, k_weight, eps, pos, q_rot,
                      k_rot, stream=None):
    """q [rows][tokens][Hq][d] and k [rows][tokens][H][d] (fp16, any strides over the first three
    dimensions; either may be None) normed per head (weights fp16 [d]; None: no norm) and rotated
    to pos (i32 [rows][tokens]; None: token t at t) into q_rot and k_rot of the same shapes."""
    n, t = (q if q is not None else k).shape[:2]
    d, hq, h = cfg.head_dim, cfg.num_q_heads, cfg.num_kv_heads
    dev = _device(stream)
    _tensor(dev, "q", q, "float16", (n, t, hq, d), True)
    _tensor(dev, "k", k, "float16", (n, t, h, d), True)
    _tensor(dev, "q_rot", q_rot, "float16", (n, t, hq, d), True)
    _tensor(dev, "k_rot", k_rot, "float16", (n, t, h, d), True)
    _tensor(dev, "q_weight", q_weight, "float16", (d,))
    _tensor(dev, "k_weight", k_weight, "float16", (d,))
    _tensor(dev, "pos", pos, "int32", (n, t))
    if table is not None and cfg.rope_kind != "none":
        _tensor(dev, "table", table, "float32", table.shape)
        if table.numel() < max_pos * d:
            raise ValueError(f"the table holds {table.numel()} values, {max_pos} positions of "
                             f"{d} channels need {max_pos * d}")
    _check(lib().fade_qk_norm_rope(ctypes.byref(cfg.c()), _ptr(table), max_pos, _heads(q),
                                   _heads(q_rot), _ptr(q_weight), _heads(k), _heads(k_rot),
                                   _ptr(k_weight), eps, _ptr(pos), n, t, _stream(stream)))


def fade_tree_ws_bytes(cfg: Config, T: int) -> int:
    """Workspace bytes of fade_tree_attention and fade_tree_commit for trees of up to T nodes."""
    n = lib().fade_tree_ws_bytes(ctypes.byref(cfg.c()), T)
    if n == 0:
        raise FadeError(FADE_ERR_INVALID_ARGUMENT, fade_last_error())
    return n


def _tree_tensors(dev, layer, q_rot, tree_k, tree_v, ws):
    cfg = layer.cfg
    T, d = q_rot.shape[1], cfg.head_dim
    kv = (cfg.batch, T, cfg.num_kv_heads, d)
    _tensor(dev, "q_rot", q_rot, "float16", (cfg.batch, T, cfg.num_q_heads, d))
    _tensor(dev, "tree_k", tree_k, "float16", kv, True)
    _tensor(dev, "tree_v", tree_v, "float16", kv, True)
    for name, t in (("the layer", layer.meta), ("ws", ws)):
        if dev is not None and t is not None and t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return T


def fade_tree_attention(layer: TieredLayer, q_rot, tree_k, tree_v, mask, n_nodes, out, lse, ws,
                        stream=None):
    """q_rot fp16 [B][T][Hq][d], tree_k / tree_v fp16 [B][T][H][d] (any strides over the first
    three dimensions), mask i64 [B][T], n_nodes i32 [B] or None -> out fp16 [B][T][Hq][d], lse
    f32 [B][T][Hq]. ws: a tensor of fade_tree_ws_bytes(cfg, T) bytes."""
    cfg = layer.cfg
    _require_codebook(layer)
    dev = _device(stream)
    T = _tree_tensors(dev, layer, q_rot, tree_k, tree_v, ws)
    _tensor(dev, "mask", mask, "int64", (cfg.batch, T))
    _tensor(dev, "n_nodes", n_nodes, "int32", (cfg.batch,))
    _tensor(dev, "out", out, "float16", q_rot.shape)
    _tensor(dev, "lse", lse, "float32", q_rot.shape[:3])
    _check(lib().fade_tree_attention(ctypes.byref(cfg.c()), ctypes.byref(layer.c), T, _ptr(q_rot),
                                     _heads(tree_k), _heads(tree_v), _ptr(mask), _ptr(n_nodes),
                                     _ptr(out), _ptr(lse), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)))


def fade_tree_commit(layer: TieredLayer, q_rot, lse, tree_k, tree_v, path, n_path, ws=None,
                     stream=None):
    """Append row b's nodes path[b][:n_path[b]] (path i32 [B][T] on the device, n_path any host
    int sequence of B lengths); H2O / EMA: their attention mass from q_rot and lse as in
    fade_tree_attention, with a workspace of fade_tree_ws_bytes(cfg, T) bytes."""
    cfg = layer.cfg
    _require_codebook(layer)
    dev = _device(stream)
    T = _tree_tensors(dev, layer, q_rot, tree_k, tree_v, ws)
    _tensor(dev, "path", path, "int32", (cfg.batch, T))
    _tensor(dev, "lse", lse, "float32", q_rot.shape[:3])
    lens = np.ascontiguousarray(n_path, np.int32)
    if lens.shape != (cfg.batch,):
        raise ValueError(f"n_path must hold {cfg.batch} lengths")
    _check(lib().fade_tree_commit(ctypes.byref(cfg.c()), ctypes.byref(layer.c), T, _ptr(q_rot),
                                  _ptr(lse), _heads(tree_k), _heads(tree_v), _ptr(path),
                                  lens.ctypes.data, _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream)))


LOGIT_TYPES = {"float16": 0, "bfloat16": 1, "float32": 2}   # fade_logit_type_t


def _logits(dev, name, t, dtype, shape):
    """A [B][T][vocab] (or [B][vocab]) tensor of logits as a fade_logits_t."""
    if t is None:
        return None
    _tensor(dev, name, t, dtype, shape, True)
    s = t.stride()
    return ctypes.byref(LogitsT(t.data_ptr(), s[0], s[1] if len(s) == 3 else 0))


def _pointer(dev, name, t, dtype, shape):
    """The address of a contiguous tensor (None: NULL)."""
    if t is None:
        return None
    _tensor(dev, name, t, dtype, shape)
    return t.data_ptr()


def fade_tree_verify(cfg: Config, parents, n_nodes, tokens, target, target_root, draft, draft_root,
                     temperature, u, noise, path, n_path, next_token, stream=None):
    """Which drafted tokens are kept: parents, tokens i32 [B][T], n_nodes i32 [B] or None; target
    [B][T][vocab] logits after every node, target_root [B][vocab] after the last cached token (None:
    node 0 is certain); draft, draft_root: the drafter's, of the same type (None: drafts without
    probabilities). temperature f32 [B] or None, u f32 [B][T] (None: greedy), noise f32 [B][vocab] or
    None -> path i32 [B][T], n_path i32 [B], next_token i32 [B]."""
    if target is None or parents is None or target.dim() != 3 or parents.dim() != 2:
        raise ValueError("target must be [rows][nodes][vocabulary], parents [rows][nodes]")
    B, T = cfg.batch, parents.shape[1]
    V = target.shape[2]
    dev = _device(stream)
    dtype = str(target.dtype).removeprefix("torch.")
    if dtype not in LOGIT_TYPES:
        raise ValueError(f"logits must be float16, bfloat16 or float32, not {dtype}")
    nodes, row, rows, vocab = (B, T), (B,), (B, T, V), (B, V)
    _check(lib().fade_tree_verify(
        ctypes.byref(cfg.c()), T, V, LOGIT_TYPES[dtype],
        _pointer(dev, "parents", parents, "int32", nodes),
        _pointer(dev, "n_nodes", n_nodes, "int32", row),
        _pointer(dev, "tokens", tokens, "int32", nodes),
        _logits(dev, "target", target, dtype, rows),
        _logits(dev, "target_root", target_root, dtype, vocab),
        _logits(dev, "draft", draft, dtype, rows),
        _logits(dev, "draft_root", draft_root, dtype, vocab),
        _pointer(dev, "temperature", temperature, "float32", row),
        _pointer(dev, "u", u, "float32", nodes), _pointer(dev, "noise", noise, "float32", vocab),
        _pointer(dev, "path", path, "int32", nodes), _pointer(dev, "n_path", n_path, "int32", row),
        _pointer(dev, "next_token", next_token, "int32", row), _stream(stream)))


def fade_prompt_ws_bytes(cfg: Config, n_q: int, n_kv: int) -> int:
    """Workspace bytes of fade_prompt_attention and fade_prompt_mass for up to n_q queries and n_kv
    tokens a row."""
    n = lib().fade_prompt_ws_bytes(ctypes.byref(cfg.c()), n_q, n_kv)
    if n == 0:
        raise FadeError(FADE_ERR_INVALID_ARGUMENT, fade_last_error())
    return n


_INT32 = np.dtype(np.int32)


def _host_lens(name, x, rows):
    """HOST i32 lengths as the bytes of a C array (None: NULL)."""
    if x is None:
        return None
    lens = np.ascontiguousarray(x)
    if lens.shape != (rows,):
        raise ValueError(f"{name} must hold {rows} lengths")
    if lens.dtype != _INT32:
        x, lens = lens, lens.astype(_INT32)
        if not (lens == x).all():   # wider integers, fractions
            raise ValueError(f"{name} must be 32-bit integers")
    return lens.tobytes()


def _i32(x):
    """An integer of any size as the 32-bit one that the prompt calls treat alike (no prompt has so many
    tokens; ctypes would take it modulo 2^32)."""
    return x if 0 <= x < 2 ** 31 else max(-1, min(x, 2 ** 31 - 1))


def _prompt_ws(cfg, dev, n_q, n_kv, q, ws, stream):
    if ws is None:   # of the stream's own memory: it is given back before the kernels have run
        with _torch.cuda.stream(stream):
            return _torch.empty(fade_prompt_ws_bytes(cfg, n_q, n_kv), dtype=_torch.uint8,
                                device=q.device)
    if not ws.is_contiguous() or (dev is not None and ws.get_device() != dev):
        raise ValueError("ws must be contiguous and on the current CUDA device")
    return ws


def fade_prompt_attention(cfg: Config, q, k, v, out, lse=None, q_len=None, kv_len=None, n_sink=0,
                          window=0, ws=None, status=None, stream=None):
    """Causal attention of q [B][n_q][Hq][d] over k and v [B][n_kv][H][d] (fp16, any strides over the
    first three dimensions) into out (like q) and lse (f32 [B][n_q][Hq], optional). A row's queries are
    the last q_len[b] of its kv_len[b] tokens (host integers; None: all). window > 0: a query sees the
    last ``window`` tokens and the first ``n_sink``. ws: fade_prompt_ws_bytes (made here when not
    given); status: a layer's status words."""
    dev = _device(stream)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [rows][tokens][heads][channels]")
    B, n_q, n_kv = cfg.batch, q.shape[1], k.shape[1]
    shape, kv = (B, n_q, cfg.num_q_heads, cfg.head_dim), (B, n_kv, cfg.num_kv_heads, cfg.head_dim)
    hq, ho = _checked_heads(dev, "q", q, shape), _checked_heads(dev, "out", out, shape)
    hk, hv = _checked_heads(dev, "k", k, kv), _checked_heads(dev, "v", v, kv)
    _tensor(dev, "lse", lse, "float32", shape[:3])
    if status is not None:
        _tensor(dev, "status", status, "int32", (STATUS_WORDS,))
    ws = _prompt_ws(cfg, dev, n_q, n_kv, q, ws, stream)
    _check(lib().fade_prompt_attention(
        ctypes.byref(cfg.c()), hq, hk, hv, n_q, n_kv, _host_lens("q_len", q_len, B),
        _host_lens("kv_len", kv_len, B), _i32(n_sink), _i32(window), ho,
        None if lse is None else lse.data_ptr(), None if status is None else status.data_ptr(),
        ws.data_ptr(), ws.nbytes, _stream(stream)))


def fade_prompt_mass(cfg: Config, q, k, lse, mass, q_len=None, kv_len=None, n_sink=0, window=0,
                     accumulate=False, ws=None, status=None, stream=None):
    """Column sums of fade_prompt_attention's probabilities, from the lse it left: mass f32
    [B][H][n_kv] (accumulate: added to)."""
    dev = _device(stream)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [rows][tokens][heads][channels]")
    B, H, n_q, n_kv = cfg.batch, cfg.num_kv_heads, q.shape[1], k.shape[1]
    shape = (B, n_q, cfg.num_q_heads, cfg.head_dim)
    hq = _checked_heads(dev, "q", q, shape)
    hk = _checked_heads(dev, "k", k, (B, n_kv, H, cfg.head_dim))
    if lse is None or mass is None:
        raise ValueError("lse and mass are needed")
    _tensor(dev, "lse", lse, "float32", shape[:3])
    _tensor(dev, "mass", mass, "float32", (B, H, n_kv))
    if status is not None:
        _tensor(dev, "status", status, "int32", (STATUS_WORDS,))
    ws = _prompt_ws(cfg, dev, n_q, n_kv, q, ws, stream)
    _check(lib().fade_prompt_mass(
        ctypes.byref(cfg.c()), hq, hk, n_q, n_kv, _host_lens("q_len", q_len, B),
        _host_lens("kv_len", kv_len, B), _i32(n_sink), _i32(window), lse.data_ptr(),
        int(bool(accumulate)), mass.data_ptr(), None if status is None else status.data_ptr(),
        ws.data_ptr(), ws.nbytes, _stream(stream)))


def fade_attention_tiled(cfg: Config) -> bool:
    """Whether decode attention for ``cfg`` runs the tensor-core kernel, whose launch is
    scheduled from every row's count of ATTN_TILE_TOKENS-token middle tiles (the host mirror
    at the call), so that a captured call stays valid only while those counts are unchanged."""
    r = lib().fade_attention_tiled(ctypes.byref(cfg.c()))
    if r < 0:
        raise FadeError(FADE_ERR_INVALID_ARGUMENT, fade_last_error())
    return bool(r)


def fade_tier_counts(layer: TieredLayer) -> np.ndarray:
    """Per-row (sinks, middle, recent) token counts from the host mirror: i32 [B][3]."""
    out = np.zeros((layer.cfg.batch, 3), np.int32)
    _check(lib().fade_tier_counts(ctypes.byref(layer.cfg.c()), ctypes.byref(layer.c),
                                  out.ctypes.data))
    return out
