"""Batch-invariant DiT AdaLN final modulation (``norm_out``) for GB300.

The operator (RL-Kernel PR 538 "final_adaln_out", section "What"):

    scale, shift = (SiLU(temb) @ W^T + b).chunk(2)      # 3072 -> 6144
    out = LayerNorm(x, eps=1e-6, no affine) * (1 + scale) + shift

with the autocast rounding points of miles_diffusion PR 108 (fp32 LayerNorm,
(1 + scale) rounded once to bf16, fp32 modulation, one bf16 store), and its
backward with token sums in a fixed 32-way tree.

Around it stand the operators of a training step or a rollout that feed it and
take its gradients on: the norm of queries and keys with the position rotation,
the embedding lookup and its gradient, the global gradient norm and clipping.

The compute lives in hand-written sm_103a CUDA kernels behind a C ABI
(``include/adaln.h`` and, for the operators around the norm,
``include/adaln_ops.h``; both built into ``libadaln.so``).  ``binding`` has the
same entry-point names for PyTorch tensors: a thin ctypes layer over the first
header, a compiled marshalling module (``csrc/marshal.cpp``) over the second.
``synth`` draws seeded synthetic inputs.  Importing this package loads nothing; the binding loads
the library on first use and fails loudly if it is missing.
"""

__all__ = ["binding", "synth"]
