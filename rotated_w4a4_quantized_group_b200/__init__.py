"""ConvRot W4A4 quantized linear for NVIDIA B200 (sm_100a).

The computation lives in libck.so (C ABI in include/ck.h); ``ck`` is its thin
Python binding and ``workloads`` draws the seeded synthetic inputs.
"""
__all__ = ["ck", "workloads", "ck_rotate_quant", "ck_w4a4_linear", "ck_unpack_w4",
           "ck_quant_fp4", "ck_dequant_fp4", "ck_fp4_linear", "ck_fp4_expert_linear"]


def __getattr__(name):
    if name.startswith("ck_") and name in __all__:
        from . import ck
        return getattr(ck, name)
    raise AttributeError(name)
