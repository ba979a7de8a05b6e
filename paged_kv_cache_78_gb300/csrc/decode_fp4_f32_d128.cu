#include "decode_fp4_inst.cuh"

PA_DEFINE_DECODE_FP4_UNIT(float, f32, 128)
