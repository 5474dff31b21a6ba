"""Fused linear cross-entropy for GB300 (sm_103a): a thin binding over ``libflce.so``.

The library computes the next-token cross-entropy of ``hidden @ weight.T`` (with
an optional bias, logit scale and soft cap), forward and backward, without
materialising the (tokens x vocab) logits.  It also holds the operators on either
side of that head: the residual addition and root-mean-square norm before it
(forward, backward, 8-bit output), the global norm and clipping of the gradients
after it, and the penalties, biases and masks on its logits when it answers; and
those that lead from one token to the next: the embedding of the ids with its
gradient, the head's logits from a weight held in 4 bits, and the choice of a token.
See ``include/flce.h``.
"""
from .api import (  # noqa: F401
    ForwardResult, LinearCrossEntropy, flce_backward, flce_forward, flce_forward_backward, flce_read_device_status,
    flce_status_string, flce_workspace_size, linear_cross_entropy, make_problem, scale_gradient,
)
from .head_ops import (  # noqa: F401
    AddRmsNorm, AddRmsNormFp8Result, AddRmsNormGrads, AddRmsNormResult, ProcessedLogits, add_rms_norm, clip_grad_norm_,
    flce_add_rms_norm, flce_add_rms_norm_backward, flce_add_rms_norm_fp8, grad_norm, process_logits,
)
from .token_ops import (  # noqa: F401
    Embedding, MxFp4, SampledTokens, embedding, flce_embedding, flce_embedding_backward, mxfp4_dequantize, mxfp4_logits,
    mxfp4_quantize, sample_tokens,
)
