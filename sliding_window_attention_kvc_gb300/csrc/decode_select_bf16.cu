// Decode over selected blocks: bf16 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_EXT_BF16(kvc::kExtSelect)
