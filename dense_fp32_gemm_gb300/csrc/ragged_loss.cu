// ragged_loss.cu -- ragged_kernel on BF16 and F16 operands with the epilogues of
// the loss over a vocabulary.
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

extern const FormEntry kFormsLoss[] = {
    SGEMM_GB300_FORM(kLse, 64, 1),   SGEMM_GB300_FORM(kLse, 128, 1),
    SGEMM_GB300_FORM(kLse, 256, 1),  SGEMM_GB300_FORM(kLse, 256, 2),
    SGEMM_GB300_FORM(kGrad, 64, 1),  SGEMM_GB300_FORM(kGrad, 128, 1),
    SGEMM_GB300_FORM(kGrad, 256, 1), SGEMM_GB300_FORM(kGrad, 256, 2),
    SGEMM_GB300_FORM(kLseFew, 16, 1), SGEMM_GB300_FORM(kGradFew, 16, 1),
    SGEMM_GB300_FORM(kLseFew, 32, 1), SGEMM_GB300_FORM(kGradFew, 32, 1),
    SGEMM_GB300_FORM(kLseFew, 64, 1), SGEMM_GB300_FORM(kGradFew, 64, 1),
};
extern const int kNumFormsLoss = sizeof(kFormsLoss) / sizeof(kFormsLoss[0]);

}  // namespace ragged
}  // namespace sgemm_gb300
