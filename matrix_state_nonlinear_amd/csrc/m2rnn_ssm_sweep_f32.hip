// The fp32-input instances of the sweep, in a file of their own to compile in parallel.
#define M2RNN_SSM_F32
#include "m2rnn_ssm_sweep.hip"
