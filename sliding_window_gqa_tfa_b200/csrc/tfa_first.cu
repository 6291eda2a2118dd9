// tfa_first.cu -- the kernels for attention with a sliding window and first
// tokens that stay visible, instantiated apart from the others (they compile
// side by side); tfa.cu prepares and launches them.
#include "tfa_bwd.cuh"
#include "tfa_first.h"
#include "tfa_kernel.cuh"

namespace tfa {
namespace {

template <int D, bool PK>
const void *forward(bool km, int mode) {
#define TFA_MODE(M) (km ? reinterpret_cast<const void *>(tfa_prefill_kernel<D, true, M, kLayoutFirst, PK>) \
                        : reinterpret_cast<const void *>(tfa_prefill_kernel<D, false, M, kLayoutFirst, PK>))
    return mode == kModePlain ? TFA_MODE(kModePlain) : mode == kModeLse ? TFA_MODE(kModeLse) : TFA_MODE(kModeSoftcap);
#undef TFA_MODE
}

}  // namespace

const void *first_forward_kernel(int D, bool key_mask, int mode, bool packed) {
    if (D == 128) return packed ? forward<128, true>(key_mask, mode) : forward<128, false>(key_mask, mode);
    return packed ? forward<64, true>(key_mask, mode) : forward<64, false>(key_mask, mode);
}

const void *first_backward_kernel(int D, bool key_mask, bool keys) {
#define TFA_PICK(D_, KM_)                                                                      \
    (keys ? reinterpret_cast<const void *>(bwd::dkv_kernel<D_, KM_, true>)                     \
          : reinterpret_cast<const void *>(bwd::dq_kernel<D_, KM_, true>))
    if (D == 128) return key_mask ? TFA_PICK(128, true) : TFA_PICK(128, false);
    return key_mask ? TFA_PICK(64, true) : TFA_PICK(64, false);
#undef TFA_PICK
}

const void *first_sum_parts_kernel(int D) {
    return D == 128 ? reinterpret_cast<const void *>(bwd::sum_parts_kernel<128>)
                    : reinterpret_cast<const void *>(bwd::sum_parts_kernel<64>);
}

}  // namespace tfa
