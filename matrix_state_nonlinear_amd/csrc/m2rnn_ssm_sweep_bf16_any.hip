// The sweep's instances for bf16 inputs, any alignment and width.
#define M2RNN_SSM_IN uint16_t
#define M2RNN_SSM_VEC false
#define M2RNN_SSM_NAME launch_ssm_sweep_bf16_any
#include "m2rnn_ssm_sweep.hip"
