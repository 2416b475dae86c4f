// ragged_dense.cu -- ragged_kernel on BF16 and F16 operands of one group.
#include "ragged_launch.cuh"

namespace sgemm_gb300 {
namespace ragged {

extern const FormEntry kFormsDense[] = {
    SGEMM_GB300_FORM(kDense, 16, 1),  SGEMM_GB300_FORM(kDense, 32, 1),
    SGEMM_GB300_FORM(kDense, 64, 1),  SGEMM_GB300_FORM(kDense, 128, 1),
    SGEMM_GB300_FORM(kDense, 256, 1), SGEMM_GB300_FORM(kDense, 256, 2),
};
extern const int kNumFormsDense = sizeof(kFormsDense) / sizeof(kFormsDense[0]);

}  // namespace ragged
}  // namespace sgemm_gb300
