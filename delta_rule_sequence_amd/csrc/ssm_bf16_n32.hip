// ssm_bf16_n32.hip - the state space scan with N = 32 on bf16 tensors
#include "prism_ssm_launch.h"
namespace prism { namespace host {
PRISM_SSM_UNIT(ssm_bf16_n32, bf16_t, 32)
} }
