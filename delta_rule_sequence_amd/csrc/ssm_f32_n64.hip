// ssm_f32_n64.hip - the state space scan with N = 64 on f32 tensors
#include "prism_ssm_launch.h"
namespace prism { namespace host {
PRISM_SSM_UNIT(ssm_f32_n64, float, 64)
} }
