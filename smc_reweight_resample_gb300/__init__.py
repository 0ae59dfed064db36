"""GB300-native speculative-decoding verify, SMC-SD reweight / resample and PACER stop rule, with what stands around them: the paged
cache, attention of drafts and trees, logits, beam search and a draft's distillation.

The compute path is the CUDA library ``libsmcsd.so`` (C ABI in ``include/smcsd.h``); the
functions exported here are its ctypes binding (``_binding``), loaded on first use. Build the
library with ``smc_reweight_resample_gb300.build.build()``. ``synth`` holds the seeded input
generators.
"""
_API = {
    "sd_verify", "smc_reweight", "smc_ess_resample", "kv_pagetable_remap", "pacer_block_stop",
    "smc_step", "Workspace", "workspace_size", "check_status", "status_string", "SMCSDError",
    "load", "OP_SD_VERIFY", "OP_SMC_REWEIGHT", "OP_SMC_STEP", "OP_ESS_RESAMPLE",
    "OP_PAGETABLE_REMAP", "OP_PACER_BLOCK_STOP", "LIB_PATH",
    "kv_slot_map", "kv_append", "tree_mask", "tree_attention", "logits_process",
    "TreeAttentionWorkspace", "OP_KV_SLOT_MAP", "OP_KV_APPEND", "OP_TREE_MASK", "OP_LOGITS_PROCESS",
    "beam_select", "state_reorder", "kv_fork", "kv_free", "kv_compact", "kv_copy_pages", "distill_loss",
    "OP_BEAM_SELECT", "OP_STATE_REORDER", "OP_KV_FORK", "OP_KV_COMPACT", "OP_DISTILL_LOSS",
}

__all__ = sorted(_API)


def __getattr__(name):
    if name in _API:
        from . import _binding

        value = globals()[name] = getattr(_binding, name)  # found here from now on
        return value
    raise AttributeError(name)
