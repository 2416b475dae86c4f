// ragged_f32.cu -- ragged_kernel on FP32 operands (three BF16 parts each).
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

extern const FormEntry kFormsF32[] = {
    SGEMM_GB300_FORM(kF32, 16, 1),
    SGEMM_GB300_FORM(kF32, 32, 1),
    SGEMM_GB300_FORM(kF32, 64, 1),
    SGEMM_GB300_FORM(kF32, 128, 1),
};
extern const int kNumFormsF32 = sizeof(kFormsF32) / sizeof(kFormsF32[0]);

}  // namespace ragged
}  // namespace sgemm_gb300
