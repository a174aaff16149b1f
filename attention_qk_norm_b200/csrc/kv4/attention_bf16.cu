// attention_bf16.cu -- attention over the 4-bit cache for bf16 activations.
#define QKN_KV4_TYPE __nv_bfloat16
#define QKN_KV4_NAME bf16
#include "attention_type.cuh"
