"""MI355X-native batched LLM sampling: fused logit processing + two-stage top-k
sampler, speculative verification, a fused LM-head Gumbel-max sampler, a 4-bit
LM head, and the pages of a key/value cache around verification.

The compute lives in libss_sampler.so (HIP, gfx950); `sampler` and `cache` are its
ctypes bindings and `workloads` builds seeded synthetic inputs.
"""
