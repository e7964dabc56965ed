// The sweep's instances for fp32 inputs.
#define M2RNN_SSM_IN float
#define M2RNN_SSM_VEC true
#define M2RNN_SSM_NAME launch_ssm_sweep_f32
#include "m2rnn_ssm_sweep.hip"
