// Decode that keeps its scores: bf16 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_EXT_BF16(kvc::kExtWeigh)
