"""MI355X-native batched LLM sampling: fused logit processing + two-stage top-k
sampler, speculative verification, a fused LM-head Gumbel-max sampler, a 4-bit
LM head, the pages of a key/value cache around verification, and rotary positions
and attention over pages of 8-bit floats.

The compute lives in libss_sampler.so (HIP, gfx950); `sampler`, `cache` and `rotary`
are its ctypes bindings and `workloads` builds seeded synthetic inputs.
"""
