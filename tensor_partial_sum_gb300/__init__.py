"""GB300-native partial-sum reduction (the reduction step of a
tensor-parallel AllReduce) behind a small C ABI.

Next to the reduction are the training operators around it: dropout joined to
the sum (``ar_reduce_dropout``) and the loss over a vocabulary split into
pieces (``ar_vocab_loss``), each with its gradient; the normalisation of the
summed residual stream (``ar_reduce_norm``) with its gradient, 8-bit
checkpoints of activations (``ar_checkpoint_pack``), and a clipped policy loss
on top of the vocabulary's (``ar_policy_loss``).

The compute path is ``libtps_ar.so`` (hand-written CUDA for sm_103a);
``tensor_partial_sum_gb300.ar`` is a ctypes binding with the same names as
the C entry points.  The first call fails loudly (RuntimeError) when the
library is not built; there is no other implementation to fall back to.
"""
from .ar import (  # noqa: F401
    AR_BF16, AR_F16, AR_F32, ARError, DTYPE_CODES, ar_check_args, ar_free, ar_init,
    ar_query, ar_reduce, ar_reduce_host, ar_reduce_variant, ar_set_option,
    ar_status_string, library_path, ArLayout, make_layout, ar_reduce_ex, ar_check_layout, ar_wire_pack,
    ar_reduce_host_noalloc, AR_NOALLOC_SCRATCH_BYTES, PreparedReduce,
    ArDropout, make_dropout, ar_reduce_dropout, ar_check_dropout, ar_reduce_dropout_grad,
    ar_reduce_dropout_grad_workspace, ArVocab, make_vocab, ar_check_vocab, ar_vocab_workspace, ar_vocab_loss,
    ar_vocab_loss_grad,
    ArNorm, make_norm, ar_reduce_norm, ar_check_norm, ar_reduce_norm_grad, ar_reduce_norm_grad_workspace,
    ArCheckpoint, AR_CHECKPOINT_BLOCK, make_checkpoint, empty_checkpoint, ar_checkpoint_pack, ar_checkpoint_unpack,
    ar_check_checkpoint, ArPolicy, make_policy, ar_check_policy, ar_policy_workspace, ar_policy_loss,
)
