// Gated linear recurrence, f16 (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_run_f16(const LinrecArgs &a, int form, bool backward, cudaStream_t st) {
    return linrec::run_form<__half>(a, form, backward, st);
}
int linrec_step_f16(const LinrecStepArgs &a, int form, cudaStream_t st) {
    return linrec::step_form<__half>(a, form, st);
}

}  // namespace trsm
