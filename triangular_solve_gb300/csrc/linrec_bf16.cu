// Gated linear recurrence, bf16, forward and single tokens (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_forward_bf16(const LinrecArgs &a, int form, cudaStream_t st) {
    return linrec::run_form<__nv_bfloat16, false>(a, form, st);
}
int linrec_step_bf16(const LinrecStepArgs &a, int form, cudaStream_t st) {
    return linrec::step_form<__nv_bfloat16>(a, form, st);
}

}  // namespace trsm
