// attention_e4m3.cu -- attention over the 4-bit cache for FP8 E4M3 activations.
#define QKN_KV4_TYPE __nv_fp8_e4m3
#define QKN_KV4_NAME e4m3
#include "attention_type.cuh"
