// Gated linear recurrence, bf16, backward (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_backward_bf16(const LinrecArgs &a, int form, cudaStream_t st) {
    return linrec::run_form<__nv_bfloat16, true>(a, form, st);
}

}  // namespace trsm
