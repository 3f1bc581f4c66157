// Gated linear recurrence, f32, forward and single tokens (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_forward_f32(const LinrecArgs &a, int form, cudaStream_t st) {
    return linrec::run_form<float, false>(a, form, st);
}
int linrec_step_f32(const LinrecStepArgs &a, int form, cudaStream_t st) {
    return linrec::step_form<float>(a, form, st);
}

}  // namespace trsm
