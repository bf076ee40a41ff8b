// Arguments of the paged-cache kernels (paged.cu), passed by value.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace nabla {

// CTAs of the paged attention: two on each of the 148 SMs (their shared memory
// allows no third).  The workspace holds two partial results of each.
constexpr int kPagedCtas = 2 * 148;
constexpr int kPagedHeads = 16;  // query heads a CTA handles together: the M of its MMAs

struct CacheArgs {
    __nv_bfloat16 *k, *v;
    int64_t k_page, k_token, k_head, v_page, v_token, v_head;  // elements
    const int32_t *table;
    int pages, page_size, heads_kv, D, seqs, width;
};

struct AppendArgs {
    CacheArgs c;
    const __nv_bfloat16 *k, *v;
    int64_t k_token, k_head, v_token, v_head;
    const int32_t *starts, *cu;
    int64_t total;
    int *status;
    int status_by_kernel;  // the first CTA writes the status word (total <= 256)
};

struct PagedArgs {
    CacheArgs c;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    int64_t q_token, q_head, o_token, o_head;
    const int32_t *lens;
    float *lse;
    int *status, *flags;  // status word; one flag a CTA
    float *part;          // [2 * CTAs][kPagedHeads][D] then [..][2]: (m, l)
    float c2;             // scale * log2(e)
    int heads, group, chunks;  // query heads, heads a key head, 16-head chunks of those
    int ctas;
};

}  // namespace nabla
