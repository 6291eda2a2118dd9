// tfa_first.h -- the kernels of tfa_first.cu, by their parameters.
#pragma once

namespace tfa {

// tfa_prefill_kernel of the first layout: head dimension, key mask, score mode, packed.
const void *first_forward_kernel(int D, bool key_mask, int mode, bool packed);
// bwd::dq_kernel, or (keys) bwd::dkv_kernel, with first tokens.
const void *first_backward_kernel(int D, bool key_mask, bool keys);

// bwd::sum_parts_kernel.
const void *first_sum_parts_kernel(int D);

}  // namespace tfa
