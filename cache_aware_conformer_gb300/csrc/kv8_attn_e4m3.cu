// The attention kernels of kv8_attn.cu for e4m3 codes, a translation unit of their own so that both compile at once.
#define KV8_ATTN_CODE 1  // CAC_KV8_E4M3
#include "kv8_attn.cu"
