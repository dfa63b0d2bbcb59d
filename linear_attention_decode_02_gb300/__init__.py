"""GB300-native Kimi Delta Attention (KDA) recurrent decode.

The decode entry points of libkda, with the C names:

    kda_recurrent_decode   T=1, split q/k/v, softplus or bounded gate
    kda_packed_decode      Kimi K3 packed QKV, T=1, bf16 state
    kda_fused_decode       short conv + SiLU, KDA step, gated RMSNorm
    kda_spec_decode        ragged speculative rows, T >= 1 tokens each
    kda_spec_verify_decode the same from a read-only state, with commit caches
    kda_packed_fused_decode fused conv + KDA + RMSNorm over ragged speculative
                           rows, with per-token conv and state checkpoints

and the operators that the attention layers and beams around them need:

    kda_rope_append        rotary positions, keys and values into a paged cache
    kda_paged_attention_decode  attention of one new token over the paged cache
    kda_beam_select        the best continuations of each request's beams
    kda_pool_move          copies, forks, clears and reorders slots of any pools
    kda_page_assign        page tables and slots of new tokens from the sequences' lengths
    kda_rope_axes_append   rotary positions on several axes, keys and values to slots of the cache
    kda_prefix_attention_decode  the attention of sequences that share prefixes, each read once

Build the library with ``python -m linear_attention_decode_02_gb300.build``.
"""

from .binding import (SCHED_AUTO, SCHED_SPLIT, SCHED_STREAM, KdaError, kda_beam_select,  # noqa: F401
                      kda_beam_select_workspace, kda_device_error, kda_fused_decode, kda_packed_decode,
                      kda_packed_fused_decode, kda_page_assign, kda_paged_attention_decode, kda_paged_attention_workspace,
                      kda_plan_schedule, kda_plan_split, kda_pool_move, kda_prefix_attention_decode,
                      kda_prefix_attention_workspace, kda_recurrent_decode, kda_rope_append,
                      kda_rope_axes_append, kda_rope_pair_axes, kda_rope_phase_steps, kda_set_schedule_override, kda_set_split_override, kda_spec_decode,
                      kda_spec_verify_decode, kda_version, library)
