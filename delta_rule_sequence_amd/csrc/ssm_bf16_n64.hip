// ssm_bf16_n64.hip - the state space scan with N = 64 on bf16 tensors
#include "prism_ssm_launch.h"
namespace prism { namespace host {
PRISM_SSM_UNIT(ssm_bf16_n64, bf16_t, 64)
} }
