"""MI355X (gfx950) prioritized-replay sum tree: HIP kernels behind a C ABI.

The public ABI is include/per.h and include/per_train.h (libper.so); per.py and
train.py are its Python bindings.
"""
from .per import (PerBuffer, PerError, load, per_add, per_capacity, per_create, per_cursor,
                  per_destroy, per_flush, per_graph_mode, per_last_error, per_max_priority, per_min, per_sample,
                  per_rank_attach,
                  per_rank_ptrs, per_rank_refresh, per_rank_workspace_bytes,
                  per_sample_padded, per_sample_philox, per_sample_rank, per_sample_uniform,
                  per_set_sample_lanes, per_size,
                  per_state_dim, per_time_next, per_total, per_tree_ptrs, per_update, per_update_add,
                  per_update_static, per_workspace_bytes)
from .train import (per_distill, per_distill_backward, per_distill_forward,
                    per_distill_workspace_bytes, per_rows_read, per_rows_write, per_rows_write_at,
                    per_scan_backward, per_scan_forward, per_scan_step, per_scan_workspace_bytes,
                    rows_alloc)

__all__ = ["PerBuffer", "PerError", "load", "per_add", "per_capacity", "per_create",
           "per_cursor", "per_destroy", "per_flush", "per_graph_mode", "per_last_error", "per_max_priority", "per_min",
           "per_rank_attach", "per_rank_ptrs", "per_rank_refresh",
           "per_rank_workspace_bytes", "per_sample", "per_sample_padded", "per_sample_philox",
           "per_sample_rank", "per_sample_uniform", "per_set_sample_lanes", "per_size", "per_state_dim", "per_time_next", "per_total", "per_tree_ptrs", "per_update",
           "per_update_add", "per_update_static",
           "per_workspace_bytes",
           "per_distill", "per_distill_backward", "per_distill_forward",
           "per_distill_workspace_bytes", "per_rows_read", "per_rows_write", "per_rows_write_at",
           "per_scan_backward", "per_scan_forward", "per_scan_step", "per_scan_workspace_bytes",
           "rows_alloc"]
