"""The hyper-connection read on AMD Instinct MI355X (gfx950).

The compute lives in libhc.so (HIP kernels behind the C ABI of include/hc.h);
`binding` marshals torch tensors to it.  `projections` does the same for
libhc_proj.so (include/hc_proj.h): the projections, router and expert products
that read the read's images; `attention` for libhc_attn.so (include/hc_attn.h): the
attention between projections.  `workloads` draws the seeded synthetic inputs.
Names are loaded on first use so that importing the package does not need the
built libraries.
"""
_BINDING_NAMES = ("hc_read", "hc_read_commit", "hc_read_bf16_lo", "hc_short_window_on", "hc_status_string", "hc_last_hip_error", "hc_dims",
                  "hc_timeouts", "hc_release", "read", "library", "HCError")

_PROJECTION_NAMES = ("project", "route", "expert_project", "expert_combine", "ProjectionError")

_ATTENTION_NAMES = ("PagedCache", "Batch", "SharedPrefix", "rotate_heads", "append_heads", "attend", "attend_shared", "AttentionError")

__all__ = list(_BINDING_NAMES + _PROJECTION_NAMES + _ATTENTION_NAMES)


def __getattr__(name):
    if name in _BINDING_NAMES:
        from . import binding
        return getattr(binding, name)
    if name in _PROJECTION_NAMES:
        from . import projections
        return getattr(projections, name)
    if name in _ATTENTION_NAMES:
        from . import attention
        return getattr(attention, name)
    raise AttributeError(name)
