"""DSpark block-drafter proposal head + greedy verify for GB300 (sm_103a).

The computation runs in libdspark.so (hand-written CUDA behind the C ABI of
include/dspark.h).  This package is its thin Python binding:

  _abi      ctypes functions with the C entry points' names
  torch_io  marshalling of torch tensors (device memory, streams) into those calls
  build     in-tree nvcc build of the library

Importing the package does not load the library; the first call does, and fails
loudly if the library has not been built.
"""
from ._abi import (DSPARK_BF16, DSPARK_F32, DSPARK_LOSS_MEAN, DSPARK_LOSS_SUM,  # noqa: F401
                   DSPARK_OK, DSparkError, check, dspark_block_norm,
                   dspark_block_norm_backward, dspark_block_norm_workspace_size,
                   dspark_clip_grads, dspark_clip_grads_workspace_size, dspark_config,
                   dspark_device_status, dspark_distill_loss,
                   dspark_distill_loss_workspace_size, dspark_embed, dspark_embed_backward,
                   dspark_embed_config, dspark_embed_workspace_size, dspark_grad,
                   dspark_head, dspark_head_loss, dspark_head_loss_workspace_size,
                   dspark_last_error, dspark_loss_config, dspark_loss_outputs,
                   dspark_norm_config, dspark_num_slots, dspark_outputs, dspark_propose,
                   dspark_propose_workspace_size, dspark_sample, dspark_sample_config,
                   dspark_sample_rows, dspark_status_string, dspark_teacher,
                   dspark_top_logits, dspark_tree_verify, dspark_verify,
                   dspark_wait_selftest, lib)
