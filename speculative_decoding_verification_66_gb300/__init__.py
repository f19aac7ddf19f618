"""GB300-native batched speculative-decoding verification.

The verification step of speculative decoding (rejection sampling of K draft
tokens against target and draft logits, truncation at the first rejection,
residual or bonus sampling; and the greedy variant) as hand-written CUDA for
sm_103a behind the C ABI in include/spec_verify.h. This package is the thin
Python binding: ``spec_verify`` and friends take torch tensors and call the
library; there is no CPU or eager fallback.

``sv_kv_append``, ``sv_kv_read`` and ``sv_chunk_attention`` (include/sv_attention.h,
libsvattention.so) are the step before it in the target model: the new
positions' keys and values go into a paged cache, 16-bit or e4m3, and their
queries attend to it.

``sv_token_logprobs`` and ``sv_distill_loss`` (include/sv_logprobs.h,
libsvlogprobs.so) stand beside it: the log probabilities, entropies and
alternatives of the tokens that a round emits, and the distillation of the
target's top alternatives into the draft model, with their gradients.
"""
from .api import (  # noqa: F401
    SV_BF16,
    SV_F32,
    SV_GREEDY,
    SV_SAMPLE,
    SV_SEQ_BAD_TOKEN,
    SV_SEQ_INDEX,
    SV_SEQ_NONFINITE,
    SV_SEQ_TIMEOUT,
    SpecVerifyError,
    launches,
    spec_verify,
    spec_verify_debug,
    spec_verify_early_exit,
    spec_verify_filtered,
    spec_verify_filtered_debug,
    spec_verify_filtered_timed,
    spec_verify_gated,
    spec_verify_host,
    spec_verify_lmhead,
    spec_verify_lmhead_debug,
    spec_verify_lmhead_gated,
    spec_verify_lmhead_timed,
    spec_verify_sharded,
    spec_verify_static,
    spec_verify_timed,
    sv_device_checks,
    sv_early_exit_workspace_bytes,
    sv_filtered_workspace_bytes,
    sv_host_staging_bytes,
    sv_lmhead_logits,
    sv_lmhead_workspace_bytes,
    sv_sharded_workspace_bytes,
    sv_philox,
    sv_workspace_bytes,
    version,
)
from .attention import (  # noqa: F401
    SV_E4M3,
    SV_F16,
    SV_SEQ_BAD_LENGTH,
    SV_SEQ_BAD_PAGE,
    SV_SEQ_OVERLAP,
    sv_chunk_attention,
    sv_chunk_attention_gated,
    sv_chunk_attention_workspace_bytes,
    sv_kv_append,
    sv_kv_read,
)
from .logprobs import (  # noqa: F401
    SV_LOGPROBS_COUNTER_BYTES,
    SV_MAX_TOP,
    SV_MAX_TOP_VOCAB,
    SV_ROW_STATS,
    SV_TAIL_BUCKET,
    SV_TAIL_RENORMALISE,
    TokenLogprobs,
    sv_distill,
    sv_distill_backward,
    sv_distill_loss,
    sv_logprobs_workspace_bytes,
    sv_token_logprobs,
    sv_token_logprobs_backward,
)
from ._lib import (  # noqa: F401
    LIB_PATH,
    LibraryMissing,
    load,
    load_attention,
    load_logprobs,
)
