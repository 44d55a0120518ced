// Decode kernels with modified scores: PAGED layout, bf16 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_SCORE_MMA(64, 1, true, false)
KVC_INST_SCORE_MMA(64, 2, true, false)
KVC_INST_SCORE_MMA(64, 4, true, false)
KVC_INST_SCORE_MMA(128, 1, true, false)
KVC_INST_SCORE_MMA(128, 2, true, false)
KVC_INST_SCORE_MMA(128, 4, true, false)
KVC_INST_SCORE_MMA(256, 1, true, false)
KVC_INST_SCORE_MMA(256, 2, true, false)
KVC_INST_SCORE_MMA(256, 4, true, false)
