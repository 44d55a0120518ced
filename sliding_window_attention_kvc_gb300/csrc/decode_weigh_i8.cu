// Decode that keeps its scores: INT8 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_EXT_I8(kvc::kExtWeigh)
