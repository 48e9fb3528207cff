"""GB300-native speculative-decoding verification.

The verification step (rejection sampling, greedy and tree verification), the
n-gram proposer, the beam selection that grows candidate trees and the
distillation of draft models from the target's logits run in hand-written sm_103a CUDA kernels behind the C ABI of include/spec_verify.h
(libspecverify.so); this package is its Python binding plus the seeded
synthetic workload generator.  Importing the package does not load the
library; the first call does, and fails loudly if it is not built.
"""
from .api import (REQ_BAD_DRAFT_LEN, REQ_BAD_LOGITS, REQ_BAD_TOKEN, SV_BF16, SV_F32,  # noqa: F401
                  BeamOutputs, DistillOutputs, TopLogits, TreeOutputs, VerifyError, VerifyOutputs,
                  alloc_outputs, spec_beam_reorder, spec_beam_select, spec_distill,
                  spec_distill_grad, spec_top_logits, spec_verify_greedy, spec_verify_sample,
                  spec_verify_tree, tree_depth, workspace)

__all__ = ["spec_top_logits", "spec_distill", "spec_distill_grad", "spec_beam_select",
           "spec_beam_reorder", "TopLogits", "DistillOutputs", "BeamOutputs",
           "spec_verify_sample", "spec_verify_greedy", "spec_verify_tree", "alloc_outputs",
           "VerifyOutputs", "TreeOutputs", "VerifyError", "workspace", "tree_depth"]
