// attention_fp16.cu -- attention over the 4-bit cache for fp16 activations.
#define QKN_KV4_TYPE __half
#define QKN_KV4_NAME fp16
#include "attention_type.cuh"
