// ragged_k16.cu -- ragged_kernel on BF16 and F16 operands.
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

extern const FormEntry kForms16[] = {
    SGEMM_GB300_FORM(k16, 16, 1),
    SGEMM_GB300_FORM(k16, 32, 1),
    SGEMM_GB300_FORM(k16, 64, 1),
    SGEMM_GB300_FORM(k16, 128, 1),
    SGEMM_GB300_FORM(k16, 256, 1),
    SGEMM_GB300_FORM(k16, 256, 2),
};
extern const int kNumForms16 = sizeof(kForms16) / sizeof(kForms16[0]);

}  // namespace ragged
}  // namespace sgemm_gb300
