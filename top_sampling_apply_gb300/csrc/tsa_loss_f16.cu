// The row-loss kernels for f16 logits.
#include "tsa_loss.cuh"

namespace tsa {

using namespace loss_detail;

const void *row_loss_kernel_f16(int mode, bool ent) {
    if (mode == 1) return reinterpret_cast<const void *>(&row_loss_kernel<1, 1, false>);
    return ent ? reinterpret_cast<const void *>(&row_loss_kernel<1, 0, true>)
               : reinterpret_cast<const void *>(&row_loss_kernel<1, 0, false>);
}
template <bool ENT>
static const void *held(int threads) {
    return threads == 128   ? reinterpret_cast<const void *>(&row_held_kernel<1, ENT, 128>)
           : threads == 256 ? reinterpret_cast<const void *>(&row_held_kernel<1, ENT, 256>)
                            : reinterpret_cast<const void *>(&row_held_kernel<1, ENT, 512>);
}
const void *row_held_kernel_f16(bool ent, int threads) { return ent ? held<true>(threads) : held<false>(threads); }
const void *row_grad_kernel_f16(bool ent) {
    return ent ? reinterpret_cast<const void *>(&row_grad_kernel<1, true>)
               : reinterpret_cast<const void *>(&row_grad_kernel<1, false>);
}

}  // namespace tsa
