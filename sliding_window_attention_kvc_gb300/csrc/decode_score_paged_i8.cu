// Decode kernels with modified scores: PAGED layout, INT8 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_SCORE_MMA(128, 1, true, true)
KVC_INST_SCORE_MMA(128, 2, true, true)
KVC_INST_SCORE_MMA(128, 4, true, true)
KVC_INST_SCORE_MMA(256, 1, true, true)
KVC_INST_SCORE_MMA(256, 2, true, true)
KVC_INST_SCORE_MMA(256, 4, true, true)
