// ssm_f32_n32.hip - the state space scan with N = 32 on f32 tensors
#include "prism_ssm_launch.h"
namespace prism { namespace host {
PRISM_SSM_UNIT(ssm_f32_n32, float, 32)
} }
