"""KDA chunked forward on GB300 (sm_103a): C-ABI library + thin ctypes binding.

The compute path is libkda.so (csrc/): hand-written CUDA kernels behind the
C ABI declared in include/kda.h.  This package only builds and loads it and
marshals arguments (kda.py).  There is no CPU fallback: without the built
library or a GPU, calls raise.  cache.py holds the tensor-level calls of the
paged 8-bit cache that a hybrid model's attention layers keep, linear.py those
of linear attention with a decay for each head, rotary.py rotary positions.
"""
import importlib
import importlib.util

from .kda import (forward, load, status_string, kda_chunk_fwd, kda_chunk_fwd_f32,  # noqa: F401
                  kda_chunk_fwd_ex, kda_chunk_fwd_host, kda_workspace_bytes,
                  kda_host_staging_bytes, kda_debug_intra, kda_build_info, kda_resolve_algo, KdaError,
                  kda_page_plan, kda_page_runs, kda_page_release, kda_cache_append,
                  kda_cache_attn, kda_cache_attn_workspace_bytes, KDA_I8, KDA_E4M3,
                  kda_linear_fwd, kda_linear_workspace_bytes, kda_linear_decode, kda_rotary,
                  KDA_OK, KDA_BF16, KDA_F32, KDA_ALGO_AUTO, KDA_ALGO_SIMT, KDA_ALGO_TC)
_CACHE = ("PagePlan", "page_plan", "page_release", "cache_append", "cache_attend")
_TENSOR = {name: "cache" for name in _CACHE} | {
    "linear_attend": "linear", "linear_decode": "linear",
    "rotary_embed": "rotary", "rotary_frequencies": "rotary"}


def __getattr__(name):
    # (these modules need torch, which the C-level binding does not: imported when asked for)
    if name in _TENSOR:
        module = importlib.import_module("." + _TENSOR[name], __name__)
        globals()[name] = getattr(module, name)
        return globals()[name]
    raise AttributeError("module %r has no attribute %r" % (__name__, name))


__all__ = ["forward", "load", "status_string", "kda_chunk_fwd", "kda_chunk_fwd_f32",
           "kda_chunk_fwd_ex", "kda_chunk_fwd_host", "kda_workspace_bytes",
           "kda_host_staging_bytes", "kda_debug_intra", "kda_build_info", "KdaError",
           "kda_page_plan", "kda_page_runs", "kda_page_release", "kda_cache_append",
           "kda_cache_attn", "kda_cache_attn_workspace_bytes", "kda_linear_fwd",
           "kda_linear_workspace_bytes", "kda_linear_decode", "kda_rotary"]
if importlib.util.find_spec("torch"):  # (a star import fetches every name listed)
    __all__ += list(_TENSOR)
