"""MI355X (gfx950) weight-only low-bit quantized Linear, static-FP8 Linear and
block-scaled FP8 operators.

The compute lives in the HIP library ``libwq.so`` (C ABI declared in
``include/wq.h`` and ``include/wq_block.h``); ``weight_only_bit_dequant_amd.wq``
is the thin ctypes binding, ``weight_only_bit_dequant_amd.block`` the
block-scaled operators.  Importing this package loads nothing; the first call into ``wq``
loads the library and raises if it is missing.
"""

__all__ = ["block", "synth", "wq"]
