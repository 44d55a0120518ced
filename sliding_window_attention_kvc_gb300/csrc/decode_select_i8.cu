// Decode over selected blocks: INT8 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_EXT_I8(kvc::kExtSelect)
