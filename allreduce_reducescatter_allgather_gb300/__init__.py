"""AllReduce, ReduceScatter and AllGather over N virtual ranks on one GB300.

N "ranks" are N device buffers in one GPU's memory.  The collectives run as
hand-written sm_103a kernels (libvc.so, C ABI in include/vc.h) that read the
N buffers with 16-byte vector loads and reduce them in registers in a fixed
order (ring, recursive halving or tree).  This package is the thin ctypes
binding with the same names as the C entry points.

Beside them, the operators of a data-parallel training step (include/vc_train.h,
training.py): the linear layer, its gradient, Newton-Schulz orthogonalisation and
the Muon step, on the tensor cores; and what a step has between and around the
linear layers (include/vc_step.h, step.py): the embedding and its gradient, the
norms around a block with its gate and residual, and gradient clipping.
"""
from ._binding import (  # noqa: F401
    BucketPlan,
    DTYPES,
    MAX_RANKS,
    OPS,
    ORDERS,
    VcError,
    Prepared,
    lib,
    prepare_all_gather,
    prepare_all_reduce,
    prepare_all_reduce_decomposed,
    prepare_reduce_scatter,
    vc_all_gather,
    vc_all_reduce,
    vc_all_reduce_decomposed,
    vc_all_reduce_decomposed_noalloc,
    vc_broadcast,
    vc_reduce,
    vc_reduce_scatter,
    vc_shard_count,
)
from .training import (  # noqa: F401
    ACTIVATIONS,
    COEFFICIENTS,
    PreparedMuon,
    PreparedOperator,
    linear_backward_workspace,
    linear_forward_workspace,
    orthogonalize_workspace,
    prepare_linear_backward,
    prepare_linear_forward,
    prepare_muon_step,
    prepare_orthogonalize,
    train_timeouts,
    vc_linear_backward,
    vc_linear_forward,
    vc_muon_step,
    vc_orthogonalize,
)
from .step import (  # noqa: F401
    ClipPlan,
    GRAD_NORMS,
    NORMS,
    block_norm_backward_workspace,
    embedding_backward_workspace,
    prepare_block_norm_backward,
    prepare_block_norm_forward,
    prepare_embedding_backward,
    prepare_embedding_forward,
    vc_block_norm_backward,
    vc_block_norm_forward,
    vc_embedding_backward,
    vc_embedding_forward,
)
