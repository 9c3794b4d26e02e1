// ssm_bf16_n128.hip - the state space scan with N = 128 on bf16 tensors
#include "prism_ssm_launch.h"
namespace prism { namespace host {
PRISM_SSM_UNIT(ssm_bf16_n128, bf16_t, 128)
} }
