// Gated linear recurrence, bf16 (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_run_bf16(const LinrecArgs &a, int form, bool backward, cudaStream_t st) {
    return linrec::run_form<__nv_bfloat16>(a, form, backward, st);
}
int linrec_step_bf16(const LinrecStepArgs &a, int form, cudaStream_t st) {
    return linrec::step_form<__nv_bfloat16>(a, form, st);
}

}  // namespace trsm
