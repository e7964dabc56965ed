// The sweep's instances for fp32 inputs, any alignment and width.
#define M2RNN_SSM_IN float
#define M2RNN_SSM_VEC false
#define M2RNN_SSM_NAME launch_ssm_sweep_f32_any
#include "m2rnn_ssm_sweep.hip"
