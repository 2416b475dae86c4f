// ragged_i8.cu -- ragged_kernel on 8-bit integer operands.
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

extern const FormEntry kFormsI8[] = {
    SGEMM_GB300_FORM(kI8, 16, 1),
    SGEMM_GB300_FORM(kI8, 32, 1),
    SGEMM_GB300_FORM(kI8, 64, 1),
    SGEMM_GB300_FORM(kI8, 128, 1),
    SGEMM_GB300_FORM(kI8Wide, 256, 1),
    SGEMM_GB300_FORM(kI8Wide, 256, 2),
};
extern const int kNumFormsI8 = sizeof(kFormsI8) / sizeof(kFormsI8[0]);

}  // namespace ragged
}  // namespace sgemm_gb300
