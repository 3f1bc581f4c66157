// Gated linear recurrence, f32 (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_run_f32(const LinrecArgs &a, int form, bool backward, cudaStream_t st) {
    return linrec::run_form<float>(a, form, backward, st);
}
int linrec_step_f32(const LinrecStepArgs &a, int form, cudaStream_t st) {
    return linrec::step_form<float>(a, form, st);
}

}  // namespace trsm
