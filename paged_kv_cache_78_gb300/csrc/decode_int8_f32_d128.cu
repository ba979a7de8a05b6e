#include "decode_int8_inst.cuh"

PA_DEFINE_DECODE_INT8_UNIT(float, f32, 128)
