#include "decode_int8_inst.cuh"

PA_DEFINE_DECODE_INT8_UNIT(__nv_bfloat16, bf16, 128)
