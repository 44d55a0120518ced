// Decode kernels with modified scores: RING and SINK_RING layouts, INT8 cache (tensor cores).
#include "decode_inst.cuh"
KVC_INST_SCORE_MMA(128, 1, false, true)
KVC_INST_SCORE_MMA(128, 2, false, true)
KVC_INST_SCORE_MMA(128, 4, false, true)
KVC_INST_SCORE_MMA(256, 1, false, true)
KVC_INST_SCORE_MMA(256, 2, false, true)
KVC_INST_SCORE_MMA(256, 4, false, true)
