// Gated linear recurrence, f16, forward and single tokens (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_forward_f16(const LinrecArgs &a, int form, cudaStream_t st) {
    return linrec::run_form<__half, false>(a, form, st);
}
int linrec_step_f16(const LinrecStepArgs &a, int form, cudaStream_t st) {
    return linrec::step_form<__half>(a, form, st);
}

}  // namespace trsm
