"""Quantized latent-MoE expert layer for B200 (sm_100a).

The layer runs in hand-written CUDA kernels behind the C ABI declared in
``include/elq.h`` (``libelq.so``).  ``quantized_latent_moe_b200.elq`` is the
thin ctypes binding: it marshals torch tensors' device pointers and the current
CUDA stream into those calls and does nothing else.  ``ops`` binds the calls of
``include/elq_ops.h`` (8-bit rows with one scale a token, products of them, dense
and grouped by expert, and the norms around a block) in the same way.  ``synth``
holds the seeded synthetic input recipe.
"""
__all__ = ["elq", "ops", "synth"]
