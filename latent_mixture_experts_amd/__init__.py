"""latent_mixture_experts_amd -- the latent MoE layer on one MI355X (gfx950).

The compute path is the C-ABI library ``libmoe.so`` (hand-written HIP kernels
for gfx950), declared in ``include/moe.h``. This package holds:

* :mod:`.binding` -- argument marshalling from torch tensors to the C-ABI
  (the layer's calls, and beside them the 8-bit and 4-bit rows and products,
  the way into and out of expert order and the router's balance loss);
* :mod:`.build`   -- the hipcc build of ``libmoe.so``;
* :mod:`.synth`   -- seeded synthetic inputs (no arithmetic of the layer).

Importing the package loads nothing; the library is loaded on first use and
a missing or unloadable library raises immediately (there is no fallback).
"""

__all__ = ["binding", "build", "synth"]
