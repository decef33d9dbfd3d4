"""Invariant Bit Packing (IBP) for AMD Instinct MI355X.

The C ABI lives in include/ibp.h and libibp.so (HIP kernels for gfx950);
`lossless_bit_level_amd.ibp` is its ctypes binding.  The 8-bit KV page cache
(append, attention, eviction) is include/ibp_kv.h, libibp_kv.so and
`lossless_bit_level_amd.ibp_kv`, which has the calls for long and shared contexts
(include/ibp_kv_long.h, libibp_kv_long.so) as well.
"""
