"""OCTOPUS KV-cache codec for NVIDIA B200 (sm_100a): encode, fused decode attention, and a paged cache with chunk
attention and eviction.

The compute path is the C ABI in ``include/octopus.h`` (library
``liboctopus_b200.so``, built by ``build.py``); :mod:`.api` is a thin
PyTorch binding of it, :mod:`.paged` that of the paged cache. :mod:`.inputs` draws the seeded synthetic workloads.
"""

from .api import (ROUND_JOINT, ROUND_SCALAR, Cache, DeviceTables, Layout, Workspace, codebook_build,  # noqa: F401
                  decode_attn, decode_attn_workspace_bytes, encode, qjl_build, rotation_build)
from .paged import (PagedCache, RopeTable, paged_append, paged_attn, paged_attn_workspace_bytes,  # noqa: F401
                    paged_evict, paged_mass, paged_mass_workspace_bytes, paged_write, rope)
