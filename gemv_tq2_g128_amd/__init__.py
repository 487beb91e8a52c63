"""gemv_tq2_g128_amd: TQ2_0_g128 ternary matmul for AMD MI355X (gfx950).

* ``csrc/``   -- the HIP kernels and the C ABI (``include/tq2.h``), built into
  ``libtq2.so`` by ``python -m gemv_tq2_g128_amd.build``;
* ``tq2``     -- the Python binding (``from gemv_tq2_g128_amd import tq2``);
  importing it raises if the library has not been built;
* ``q4``      -- 4-bit matrix-vector products with group scales (``include/tq2_q4.h``);
* ``attn``    -- the paged key/value cache: appending with rotation, and
  attention over it (``include/tq2_attn.h``);
* ``moe``     -- mixtures of experts: the router, and the chosen experts'
  feed-forward on 4-bit or ternary weights (``include/tq2_moe.h``);
* ``sampling`` -- the next token from logits: temperature, top-k, min-p and
  top-p (``include/tq2_sample.h``).
"""
