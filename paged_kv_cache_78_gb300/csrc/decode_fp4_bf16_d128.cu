#include "decode_fp4_inst.cuh"

PA_DEFINE_DECODE_FP4_UNIT(__nv_bfloat16, bf16, 128)
