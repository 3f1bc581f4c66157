// Gated linear recurrence, f32, backward (see linrec.cuh).
#include "linrec.cuh"

namespace trsm {

int linrec_backward_f32(const LinrecArgs &a, int form, cudaStream_t st) {
    return linrec::run_form<float, true>(a, form, st);
}

}  // namespace trsm
