"""Per-rank hot path of ZeRO-3 intra-layer partitioning on MI355X (gfx950).

Each parameter is flattened, padded to a multiple of N_d and split into N_d
contiguous 1D shards; gradients of N_d virtual ranks are reduced into the
owned shard in fixed rank order (fp32); a fused mixed-precision Adam step
updates the fp32 master and moments and writes the bf16 working copy; a full
parameter is gathered and unpadded from its N_d shards just before compute.
The global norm of the gradients, sharded or not, and updates clipped by it
stay on the device.
All work runs in the HIP kernels of libzsp.so behind the C ABI in
include/zsp.h; this package is its thin ctypes binding.
"""
from .binding import (  # noqa: F401
    ALL_RANKS, BF16, F32, GRADS_FULL, GRADS_SHARD, MAX_RANKS, NORM_L2, NORM_MAX, SRC_ACC,
    SRC_MASTER, SRC_WORK, GatherList, Plan, Schedule, TensorList, ZspError, clip_combine,
    clip_many, clip_record, clip_values, last_error, norm_many, norm_workspace, partition,
    zsp_adam_step, zsp_adam_step_clip, zsp_adam_step_clip_params, zsp_adam_step_params,
    zsp_bind_state, zsp_checkpoint_load, zsp_checkpoint_read_host, zsp_checkpoint_save,
    zsp_checkpoint_write_host, zsp_clip_combine, zsp_clip_many, zsp_destroy, zsp_gather,
    zsp_gather_list_create, zsp_gather_list_destroy, zsp_gather_list_run, zsp_gather_many,
    zsp_gather_many_noalloc, zsp_gather_range, zsp_grad_norm, zsp_grad_norm_params,
    zsp_load_params, zsp_norm_many, zsp_norm_workspace, zsp_partition, zsp_plan_info,
    zsp_plan_tensor, zsp_reduce_adam_step, zsp_reduce_adam_step_clip,
    zsp_reduce_adam_step_clip_params, zsp_reduce_adam_step_params, zsp_reduce_norm,
    zsp_reduce_shard, zsp_reduce_shard_norm, zsp_reduce_shard_norm_params,
    zsp_reduce_shard_params, zsp_sched_acquire, zsp_sched_bind, zsp_sched_create,
    zsp_sched_destroy, zsp_sched_info, zsp_sched_release, zsp_sched_reset, zsp_sched_set_engine,
    zsp_tensor_list_clip, zsp_tensor_list_create, zsp_tensor_list_destroy, zsp_tensor_list_norm,
)
