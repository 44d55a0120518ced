// Decode kernels with modified scores: RING and SINK_RING layouts, bf16 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_SCORE_MMA(64, 1, false, false)
KVC_INST_SCORE_MMA(64, 2, false, false)
KVC_INST_SCORE_MMA(64, 4, false, false)
KVC_INST_SCORE_MMA(128, 1, false, false)
KVC_INST_SCORE_MMA(128, 2, false, false)
KVC_INST_SCORE_MMA(128, 4, false, false)
KVC_INST_SCORE_MMA(256, 1, false, false)
KVC_INST_SCORE_MMA(256, 2, false, false)
KVC_INST_SCORE_MMA(256, 4, false, false)
