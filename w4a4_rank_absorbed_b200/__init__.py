"""B200-native (sm_100a) SVDQuant W4A4 linear layer, with its 8-bit integer form and group norm.

    svdq      -- binding of the C ABI (include/svdq.h) of libsvdq.so
    layer     -- SVDQLinear: packed layer, forward = quantize_act + linear; W8A8Linear, GroupNorm
    calib     -- offline smoothing / SVD / residual decomposition (float64, host)
    synth     -- seeded synthetic workloads
    build     -- nvcc build of libsvdq.so (in-tree)
"""
__all__ = ["svdq", "layer", "calib", "synth", "build"]
