"""GB300-native selective state-space scan: a C-ABI CUDA library (``libssm.so``)
and its thin Python binding.

Entry points (same names as in ``include/ssm.h``): ``ssm_scan_fwd``,
``ssm_scan_bwd``, ``ssm_scan_fwd_host``, ``ssd_chunked_fwd``, ``ssd_chunked_bwd``, ``ssm_decode_step``, ``ssd_mamba3_fwd``,
``ssm_decode_step_mamba3``, ``ssd_mamba3_mimo_fwd``, ``ssm_decode_step_mamba3_mimo``,
``ssm_scan_workspace_bytes``, ``ssm_scan_bwd_workspace_bytes``,
``ssm_last_device_status``; around the mixers: ``ssm_add_rmsnorm_fwd``,
``ssm_add_rmsnorm_e4m3_fwd``, ``ssm_add_rmsnorm_bwd`` (RMS norm with the residual's
addition), ``ssm_linrec_fwd``, ``ssm_linrec_bwd`` (gated linear recurrence), ``ssm_vocab_ce_fwd``,
``ssm_vocab_ce_bwd`` (cross entropy over a vocabulary).  The library is loaded on first call; building it is
``state_space_model_selective_gb300.build.build()``.
"""
from .binding import (EXPORTS, SSMError, lib, ssd_chunked_bwd,  # noqa: F401
                      ssm_add_rmsnorm_bwd, ssm_add_rmsnorm_bwd_workspace_bytes,
                      ssm_add_rmsnorm_e4m3_fwd, ssm_add_rmsnorm_fwd, ssm_linrec_bwd,
                      ssm_linrec_bwd_workspace_bytes, ssm_linrec_checkpoint_bytes,
                      ssm_linrec_fwd, ssm_linrec_workspace_bytes,
                      ssd_chunked_checkpoint_bytes,
                      ssd_chunked_bwd_workspace_bytes, ssd_chunked_fwd, ssd_mamba3_fwd,
                      ssd_mamba3_mimo_fwd, ssm_abi_version, ssm_decode_step,
                      ssm_decode_step_mamba3, ssm_decode_step_mamba3_mimo,
                      ssm_last_device_status, ssm_scan_bwd, ssm_scan_bwd_workspace_bytes,
                      ssm_scan_checkpoint_bytes, ssm_scan_fwd, ssm_scan_fwd_host,
                      ssm_scan_fwd_host_workspace_bytes,
                      ssm_scan_workspace_bytes, ssm_vocab_ce_bwd,
                      ssm_vocab_ce_bwd_workspace_bytes, ssm_vocab_ce_fwd,
                      ssm_vocab_ce_workspace_bytes, status_string)
