"""MI355X-native Kimi Delta Attention (KDA) forward operator.

The operator lives in libkda.so (HIP kernels for gfx950 behind the C ABI of
include/kda.h); `gated_delta_rule_10_amd.kda` is its Python binding and
`gated_delta_rule_10_amd.inputs` draws seeded synthetic inputs. The softmax
attention of the layers between KDA layers, and its paged key/value cache
(include/kda_attn.h), are bound in `gated_delta_rule_10_amd.attn`.
"""

__all__ = ["kda_chunk_fwd", "kda_decode_step", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd_ex",
           "kda_decode_step_ex", "kda_chunk_fwd_ex_noalloc", "kda_abi_version", "kda_status_string", "KDAError"]
_ATTN = ["kda_attn_fwd", "kda_kv_write", "kda_kv_read", "kda_attn_cache_fwd", "kda_attn_cache_fwd_workspace_size"]
__all__ += _ATTN


def __getattr__(name):
    # the bindings import torch; load them only when one of their names is used
    if name in _ATTN:
        from . import attn
        globals()[name] = f = getattr(attn, name)
        return f
    if name in __all__:
        from . import kda
        return getattr(kda, name)
    raise AttributeError(name)
