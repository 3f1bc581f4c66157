// Gated linear recurrence, f16, backward (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_backward_f16(const LinrecArgs &a, int form, cudaStream_t st) {
    return linrec::run_form<__half, true>(a, form, st);
}

}  // namespace trsm
