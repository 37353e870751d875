"""Falcon fast-weight updates (Fast Weight Attention) on B200 (sm_100a).

The computation lives in libfalcon.so (C ABI in include/falcon.h, CUDA
kernels in csrc/); this package is the thin ctypes binding plus the seeded
synthetic-input generator.  layer.py binds the operators of the layer around
the update: the gated recurrence and the norms.
"""
from ._lib import (DTYPES, EXPORTS, FORMS, LIB_PATH, VARIANTS, FalconError, carry_from_prefill,  # noqa: F401
                   bwd, check_decode_shapes, check_fwd_shapes, decode_step, fwd, fwd_host, fwd_masked_noalloc,
                   fwd_workspace_size, load, scratch_trim, selftest_bounded_wait, wait_timeouts)
from .layer import (NORM_MAX_D, SCAN_BLOCK, check_norm_gate_shapes, check_residual_norm_shapes,  # noqa: F401
                    check_scan_shapes, norm_gate, norm_gate_bwd, norm_gate_bwd_workspace_size, residual_norm,
                    residual_norm_bwd, residual_norm_bwd_workspace_size, scan, scan_bwd, scan_bwd_workspace_size,
                    scan_step)
