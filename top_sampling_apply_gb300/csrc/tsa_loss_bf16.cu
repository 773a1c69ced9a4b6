// The row-loss kernels for bf16 logits.
#include "tsa_loss.cuh"

namespace tsa {

namespace {

template <int MODE, bool GRAD, bool ENT>
const void *pick(int form) {
    using namespace loss_detail;
    return form == 1 ? reinterpret_cast<const void *>(&row_loss_kernel<2, MODE, GRAD, ENT>)
                     : reinterpret_cast<const void *>(&row_loss_stream_kernel<2, MODE, GRAD, ENT>);
}

}  // namespace

const void *row_loss_kernel_bf16(int mode, bool grad, bool ent, int form) {
    if (mode == 1) return pick<1, false, false>(form);
    if (grad) return ent ? pick<0, true, true>(form) : pick<0, true, false>(form);
    return ent ? pick<0, false, true>(form) : pick<0, false, false>(form);
}

const void *row_grad_kernel_bf16() { return reinterpret_cast<const void *>(&loss_detail::row_grad_kernel<2>); }

}  // namespace tsa
