"""selective_state_space_fwd_gb300 -- the fused selective scan on GB300, and the
operators around it in a language model's layer.

The compute lives in ``libssmscan.so`` (C ABI, include/ssmscan.h, hand-written
sm_103a kernels under csrc/).  This package is its Python binding plus the
seeded synthetic workloads used by the benchmark and tests.
"""
from ._binding import (Kernel, SsmError, Status, check_device_errors, chunk_count,
                       decode_step, declared_functions,
                       host_workspace_bytes, kernel_name, load, plan, scan_bwd, scan_fwd, scan_fwd_host,
                       scan_fwd_host_static, scan_fwd_split, selftest_wait_timeout, split_plan,
                       ssd_fwd, static_capacity,
                       status_string, version)
from .layers import (conv_bwd, conv_fwd, conv_step, distill_bwd, distill_fwd, embed_bwd, embed_fwd,
                     norm_bwd, norm_fwd, recur_bwd, recur_fwd, recur_step, xent_bwd, xent_fwd)
from .autograd import (causal_conv, embedding, gated_recurrence, layer_norm, linear_cross_entropy,
                       linear_distillation, selective_scan)

__all__ = ["Kernel", "SsmError", "Status", "causal_conv", "check_device_errors", "chunk_count",
           "conv_bwd", "conv_fwd", "conv_step", "decode_step", "declared_functions",
           "distill_bwd", "distill_fwd", "embed_bwd", "embed_fwd", "embedding", "gated_recurrence", "host_workspace_bytes", "kernel_name", "layer_norm", "linear_cross_entropy", "linear_distillation", "load", "norm_bwd", "norm_fwd",
           "plan", "recur_bwd", "recur_fwd", "recur_step", "scan_bwd", "scan_fwd",
           "scan_fwd_host", "scan_fwd_host_static", "scan_fwd_split", "selftest_wait_timeout",
           "selective_scan", "split_plan", "ssd_fwd",
           "static_capacity",
           "status_string", "version", "xent_bwd", "xent_fwd"]
