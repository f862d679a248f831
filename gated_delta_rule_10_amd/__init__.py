"""MI355X-native Kimi Delta Attention (KDA) forward operator.

The operator lives in libkda.so (HIP kernels for gfx950 behind the C ABI of
include/kda.h); `gated_delta_rule_10_amd.kda` is its Python binding and
`gated_delta_rule_10_amd.inputs` draws seeded synthetic inputs. The softmax
attention of the layers between KDA layers, and its paged key/value cache
(include/kda_attn.h), are bound in `gated_delta_rule_10_amd.attn`; linear
attention with one decay per head (include/kda_lin.h) in
`gated_delta_rule_10_amd.lin`, and beam search over the states of both kinds of
layer (include/kda_beam.h) in `gated_delta_rule_10_amd.beam`.
"""

__all__ = ["kda_chunk_fwd", "kda_decode_step", "kda_chunk_fwd_workspace_size", "kda_chunk_fwd_ex",
           "kda_decode_step_ex", "kda_chunk_fwd_ex_noalloc", "kda_abi_version", "kda_status_string", "KDAError"]
_ATTN = ["kda_attn_fwd", "kda_kv_write", "kda_kv_read", "kda_attn_cache_fwd", "kda_attn_cache_fwd_workspace_size"]
_LIN = ["kda_lin_chunk_fwd", "kda_lin_chunk_fwd_workspace_size", "kda_lin_decode_step"]
_BEAM = ["kda_beam_select", "kda_beam_select_workspace_size", "kda_state_reorder"]
__all__ += _ATTN + _LIN + _BEAM


def __getattr__(name):
    # the bindings import torch; load them only when one of their names is used
    if name in _ATTN + _LIN + _BEAM:
        if name in _ATTN:
            from . import attn as module
        elif name in _LIN:
            from . import lin as module
        else:
            from . import beam as module
        globals()[name] = f = getattr(module, name)
        return f
    if name in __all__:
        from . import kda
        return getattr(kda, name)
    raise AttributeError(name)
