"""MI355X (gfx950) weight-only low-bit quantized Linear, static-FP8 Linear,
block-scaled FP8 and 8-bit integer operators, and the experts' routing.

The compute lives in the HIP library ``libwq.so`` (C ABI declared in
``include/wq.h``, ``wq_block.h``, ``wq_int8.h`` and ``wq_experts.h``);
``weight_only_bit_dequant_amd.wq`` is the thin ctypes binding, ``.block`` holds
the block-scaled operators, ``.int8`` the integer ones, ``.experts`` routing.
Importing this package loads nothing; the first call into ``wq`` loads the library
and raises if it is missing.
"""

__all__ = ["block", "experts", "int8", "synth", "wq"]
