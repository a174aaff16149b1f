// attention_fp32.cu -- attention over the 4-bit cache for fp32 activations.
#define QKN_KV4_TYPE float
#define QKN_KV4_NAME fp32
#include "attention_type.cuh"
