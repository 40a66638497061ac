"""Tree conv, tree Gated DeltaNet, tree attention, token log probabilities and the
token embedding (forward and backward) for MI355X (gfx950), over a packed prefix trie.

    plan = tree_plan(parents, seg_lens, conv_width=4)   # host, once per forward
    y = tree_conv(x, w, plan)                            # [N, C]
    o = tree_gdn_scan(q, k, v, g, beta, plan)            # [N, H_v, d_v]
    o = tree_attention(q, k, v, plan)                    # [N, H_q, d]
    r = tree_logprobs(logits, tokens, plan)              # r.logp [N], r.entropy [N]
    x = tree_embedding(tokens, table)                    # [N, C]
    r = tree_linear_logprobs(x, table, tokens, plan)     # without the logits

The kernels live in libtreegdn.so (C ABI in include/tree_gdn.h); this module
only marshals torch tensors into pointers and the current HIP stream.
"""
from ._lib import (  # noqa: F401
    TokenLogprobs,
    TreeError,
    TreePlan,
    load,
    tree_attention,
    tree_attention_backward,
    tree_conv,
    tree_conv_backward,
    tree_embedding,
    tree_embedding_backward,
    tree_gdn_scan,
    tree_gdn_scan_backward,
    tree_linear_logprobs,
    tree_linear_logprobs_backward,
    tree_logprobs,
    tree_logprobs_backward,
    tree_plan,
    tree_ssd_scan,
)
