"""B200-native (sm_100a) forward pass of a DeepSeek-V3/R1 Mixture-of-Experts block.

The block runs in four C-ABI CUDA libraries (moe_router, moe_dispatch,
moe_experts, moe_combine; headers in include/); a fifth, moe_train, holds the
experts' training operators.  This package is their thin Python binding plus
the seeded input generator.
"""
from .moe import (BlockParams, BlockShape, MoEBlock, combine, dispatch_build,  # noqa: F401
                  expert_weights_struct, experts_forward, router_forward, selftest_wait)
from .training import (Checkpoint, ExpertGrads, SavedExperts, checkpoint_rows,  # noqa: F401
                       experts_training_backward, experts_training_forward, gather_rows,
                       grouped_linear, grouped_linear_dw, grouped_linear_dx, restore_rows,
                       swiglu_backward, swiglu_checkpoint, training_rows)
