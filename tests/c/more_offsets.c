/* Prints the sizes and field offsets of the normalisation, checkpoint and
 * policy structures, for the binding's mirrors of them. */
#include <stddef.h>
#include <stdio.h>

#include "ar.h"

#define SIZE(t) printf(#t " %zu\n", sizeof(t))
#define AT(t, f) printf(#t "." #f " %zu\n", offsetof(t, f))

int main(void) {
    SIZE(ar_checkpoint);
    AT(ar_checkpoint, ne0); AT(ar_checkpoint, ne1); AT(ar_checkpoint, format); AT(ar_checkpoint, codes);
    AT(ar_checkpoint, code_row_bytes); AT(ar_checkpoint, scales); AT(ar_checkpoint, scale_row_bytes);
    SIZE(ar_norm);
    AT(ar_norm, kind); AT(ar_norm, eps); AT(ar_norm, weight); AT(ar_norm, shift); AT(ar_norm, bias);
    SIZE(ar_norm_kept);
    AT(ar_norm_kept, sums); AT(ar_norm_kept, sum_row_bytes); AT(ar_norm_kept, n_sums); AT(ar_norm_kept, mean);
    AT(ar_norm_kept, rstd); AT(ar_norm_kept, checkpoint);
    SIZE(ar_policy);
    AT(ar_policy, tokens); AT(ar_policy, sequences); AT(ar_policy, offsets); AT(ar_policy, nll); AT(ar_policy, old_nll);
    AT(ar_policy, ref_nll); AT(ar_policy, advantages); AT(ar_policy, token_advantages); AT(ar_policy, mask);
    AT(ar_policy, clip_low); AT(ar_policy, clip_high); AT(ar_policy, kl_weight); AT(ar_policy, scale); AT(ar_policy, mean);
    return 0;
}
