// The kernel for few rows over a shared prefix and a sequence's own tokens, each sequence for itself:
// kv_attention.cu's, with a second page table.
#define MXQ_KV_TWO
#include "kv_attention.cu"
