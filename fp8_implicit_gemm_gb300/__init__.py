"""FP8 (e4m3) implicit-GEMM 3D convolution with a BF16 NCDHW output, and the 8-bit transformer path
(norm, gated activation and products of int8 or e4m3 codes), for one GB300 (sm_103a)."""
