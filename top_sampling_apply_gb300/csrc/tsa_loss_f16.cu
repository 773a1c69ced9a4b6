// The row-loss kernels for f16 logits.
#include "tsa_loss.cuh"

namespace tsa {

const void *row_loss_kernel_f16(int mode, bool grad, bool ent) {
    using namespace loss_detail;
    if (mode == 1) return reinterpret_cast<const void *>(&row_loss_kernel<1, 1, false, false>);
    if (grad)
        return ent ? reinterpret_cast<const void *>(&row_loss_kernel<1, 0, true, true>)
                   : reinterpret_cast<const void *>(&row_loss_kernel<1, 0, true, false>);
    return ent ? reinterpret_cast<const void *>(&row_loss_kernel<1, 0, false, true>)
               : reinterpret_cast<const void *>(&row_loss_kernel<1, 0, false, false>);
}

const void *row_held_kernel_f16(bool ent) {
    using namespace loss_detail;
    return ent ? reinterpret_cast<const void *>(&row_held_kernel<1, true>)
               : reinterpret_cast<const void *>(&row_held_kernel<1, false>);
}

const void *row_grad_kernel_f16() { return reinterpret_cast<const void *>(&loss_detail::row_grad_kernel<1>); }

}  // namespace tsa
