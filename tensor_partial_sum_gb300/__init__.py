"""GB300-native partial-sum reduction (the reduction step of a
tensor-parallel AllReduce) behind a small C ABI.

Next to the reduction are the training operators around it: dropout joined to
the sum (``ar_reduce_dropout``) and the loss over a vocabulary split into
pieces (``ar_vocab_loss``), each with its gradient.

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
)
