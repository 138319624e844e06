"""GB300-native grouped-query-attention AV decode reduction.

    out[b, q_h, d] = sum_{c < L_b} attn[b, c, q_h] * V[b, c, q_h // G, d]

computed by hand-written sm_103a kernels behind a C ABI (include/gqa_av.h),
the decode score step before it (include/gqa_qk.h):

    attn[b, c, q_h] = softmax over c < L_b of scale * q[b, q_h, :] . K[b, c, q_h // G, :]

and both fused in one pass over the KV cache (include/gqa_attn.h). Around them
for a paged cache: block tables, slots, and the norm, rotation and cache write of
a step's tokens, forks, accepted drafts and release (include/gqa_kv.h), and decode
attention over the paged cache for sequences that share prefixes
(include/gqa_prefix.h). For several new tokens a sequence: causal attention of
packed prompts and attention of drafted trees over the paged cache
(include/gqa_prompt.h).

``workloads`` (seeded inputs) imports without the CUDA library; the binding
functions below need the built library and raise ImportError without it.
"""
from . import workloads  # noqa: F401

_BINDING = ("gqa_av_decode", "gqa_av_decode_per_head", "gqa_av_decode_tuned",
            "gqa_av_decode_noalloc", "gqa_av_plan",
            "gqa_av_workspace_bytes", "gqa_av_set_workspace", "gqa_av_device_status",
            "gqa_av_status_string", "gqa_av_last_error", "GqaAvError", "MODE_AUTO",
            "MODE_PER_HEAD", "MODE_GQA", "GQA_AV_BF16", "GQA_AV_FP16",
            "gqa_qk_softmax_decode", "gqa_qk_device_status", "gqa_av_decode_paged",
            "gqa_attn_decode", "gqa_attn_plan", "gqa_attn_device_status",
            "gqa_kv_tables", "gqa_kv_norm_rope_append", "GQA_KV_F32",
            "gqa_prefix_attn_decode", "gqa_prefix_device_status",
            "gqa_prefix_release_graph_workspaces",
            "KvPools", "gqa_kv_fork", "gqa_kv_keep", "gqa_kv_release",
            "gqa_prompt_attn", "gqa_tree_attn", "gqa_prompt_device_status",
            "gqa_prompt_release_graph_workspaces")


def __getattr__(name):
    if name in _BINDING or name == "native":
        from . import _native
        return _native if name == "native" else getattr(_native, name)
    raise AttributeError(name)
