// A paged key-value cache: writing rows into its pages, and the attention of
// one new token per sequence over it.
//
// append: a copy, bounded by HBM.  One thread a 16-byte piece of the rows; the
// first threads of a CTA find the place of its tokens once for all of them, and
// every CTA looks at every border: if one does not ascend or leaves the rows given,
// none writes anything.
//
// paged attention: every cached row is read once for up to 16 query heads of its key
// head, 4 D bytes for 4 D flop and query head, so HBM bounds it (a larger group is
// cut into chunks of 16, each of which reads the rows again).  Work is cut into tiles of 64
// keys of one (sequence, key head, chunk of up to 16 query heads); the tiles of
// the whole batch form one line, which the CTAs share out evenly, so ragged
// lengths and a single long sequence balance alike.  A CTA therefore owns a
// run of tiles that may begin and end inside a sequence: what covers a
// sequence entirely is written out, the (at most two) pieces that do not go to
// the workspace as (m, l, unnormalised o), and join_kernel adds them in order.
// The cut depends on the lengths alone: the same lengths give the same bits.
//
// Inside a CTA each of the 4 warps owns 16 keys of a tile with its own
// softmax state and its own ring of 3 cp.async stages (16 keys of K and V, 8 KB
// at D = 128), so no barrier stands in the loop; warps join once per sequence.
// A warp's 16 keys x 16 heads go through m16n8k16 MMAs (heads padded to 16):
// the arithmetic is far below the tensor pipe's rate at the memory's speed,
// and unlike tcgen05 they need no shared accumulator or issuing thread between
// the ring and the softmax.  Scores, statistics and sums are float32; P
// is rounded to bf16 for its MMA, its sum is taken in front of the rounding.
#include "common.cuh"
#include "launch.cuh"
#include "paged.cuh"

namespace nabla {
namespace paged {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kKeys = 16;                  // keys a warp step
constexpr int kTileKeys = kKeys * kWarps;  // keys a tile
constexpr int kStages = 3;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kAppendTokens = 8;  // most tokens a CTA takes

// Element offsets of a token's rows in the pools, -1 for a token that is not
// written; true when that is because its place is out of range.
__device__ __forceinline__ bool find_place(const AppendArgs &a, int64_t tok, int64_t *pk, int64_t *pv) {
    int s = -1;
    int64_t i = 0;
    *pk = *pv = -1;
    if (a.cu == nullptr) {
        s = static_cast<int>(tok);
    } else if (tok >= a.cu[0] && tok < a.cu[a.c.seqs]) {
        int lo = 0, hi = a.c.seqs;  // last s with cu[s] <= tok
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= tok)
                lo = mid;
            else
                hi = mid;
        }
        s = lo;
        i = tok - a.cu[s];
    }
    if (s < 0) return false;  // of no sequence
    const int64_t p = a.starts[s] + i;
    const int64_t col = p / a.c.page_size;
    int page = -1;
    if (p >= 0 && i >= 0 && col < a.c.width) page = a.c.table[static_cast<int64_t>(s) * a.c.width + col];
    if (page < 0 || page >= a.c.pages) return true;
    const int64_t r = p - col * a.c.page_size;
    *pk = page * a.c.k_page + r * a.c.k_token;
    *pv = page * a.c.v_page + r * a.c.v_token;
    return false;
}

// kStride: a CTA takes one group of tokens after another (as the loop for everyone it cost
// 11% of 134 MB of prompts, in registers)
template <bool kStride>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendArgs a, int per_cta) {
    constexpr int U = 4;  // pieces a thread has in flight
    __shared__ int64_t place[2][kAppendTokens];
    int64_t t0 = static_cast<int64_t>(blockIdx.x) * per_cta;
    const int chunks = a.c.D / 8;                // 16-byte pieces a row
    const int row = a.c.heads_kv * chunks;       // pieces of all heads
    int n = 0;                                   // of the group, K and V
    uint4 w[U];
    int64_t at[U];  // in the page row: element offset; the token in `who`
    int who[U];
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int x = base + u * 256;
            who[u] = -1;
            if (x < n) {
                const int which = x % row, tv = x / row, j = tv >> 1, h = which / chunks, c = which % chunks;
                who[u] = tv;
                at[u] = ((tv & 1) ? h * a.c.v_head : h * a.c.k_head) + 8 * c;
                const __nv_bfloat16 *src = (tv & 1) ? a.v + (t0 + j) * a.v_token + h * a.v_head
                                                    : a.k + (t0 + j) * a.k_token + h * a.k_head;
                w[u] = __ldg(reinterpret_cast<const uint4 *>(src) + c);
            }
        }
    };
    // (with status_by_kernel the first CTA looks at the other CTAs' tokens too)
    const bool all = a.status_by_kernel && blockIdx.x == 0;
    bool crooked = a.cu != nullptr;  // until the borders have been looked at
    for (;;) {
        const int tokens = static_cast<int>(a.total - t0 < per_cta ? a.total - t0 : per_cta);
        n = tokens * row * 2;
        fetch(threadIdx.x);  // the first pieces travel while the places are looked up
        bool bad = false;
        if (threadIdx.x < (all ? static_cast<int>(a.total) : tokens)) {
            int64_t pk, pv;
            bad = find_place(a, t0 + threadIdx.x, &pk, &pv);
            if (threadIdx.x < tokens) {
                place[0][threadIdx.x] = pk;
                place[1][threadIdx.x] = pv;
            }
        }
        if (crooked) {
            crooked = false;
            for (int s = threadIdx.x; s < a.c.seqs; s += 256)
                crooked |= a.cu[s] < 0 || a.cu[s + 1] < a.cu[s] || a.cu[s + 1] > a.total;
            crooked = __syncthreads_or(crooked);
        }
        bad = __syncthreads_or(bad || crooked);
        if (threadIdx.x == 0 && a.status != nullptr) {
            if (all)
                *a.status = bad ? kDevParam : kDevOk;
            else if (bad && !a.status_by_kernel)
                atomicExch(a.status, kDevParam);
        }
        if (crooked) return;
        for (int base = threadIdx.x; base < n; base += U * 256) {
            if (base != threadIdx.x) fetch(base);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (who[u] < 0) continue;
                const int64_t p = place[who[u] & 1][who[u] >> 1];
                if (p >= 0)
                    *reinterpret_cast<uint4 *>(((who[u] & 1) ? a.c.v : a.c.k) + p + at[u]) = w[u];
            }
        }
        if constexpr (!kStride) return;
        t0 += static_cast<int64_t>(gridDim.x) * per_cta;
        if (t0 >= a.total) return;
        __syncthreads();  // the places have been read
    }
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
__device__ __forceinline__ int clean_len(const PagedArgs &a, int s, bool *bad) {
    const int n = a.lens[s];
    if (n < 0 || n > static_cast<int64_t>(a.c.width) * a.c.page_size) {
        *bad = true;
        return 0;
    }
    return n;
}
__device__ __forceinline__ int tiles_of(int len) {  // no overflow near 2^31
    return len / kTileKeys + (len % kTileKeys != 0);
}

// Tiles of the sequences in front of `s` and of all of them, by the whole CTA
// (NT threads); sums: shared, 2 * NT / 32 entries.
template <int NT>
__device__ __forceinline__ void tile_sums(const PagedArgs &a, int s, int64_t *sums, int64_t *front,
                                          int64_t *all) {
    int64_t f = 0, t = 0;
    bool bad = false;
    for (int i = threadIdx.x; i < a.c.seqs; i += NT) {
        const int n = tiles_of(clean_len(a, i, &bad));
        t += n;
        if (i < s) f += n;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        f += __shfl_xor_sync(0xffffffffu, f, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    if ((threadIdx.x & 31) == 0) {
        sums[threadIdx.x >> 5] = f;
        sums[NT / 32 + (threadIdx.x >> 5)] = t;
    }
    __syncthreads();
    *front = *all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        *front += sums[w];
        *all += sums[NT / 32 + w];
    }
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(take ? 16 : 0));
}

template <int D>
constexpr uint32_t stage_bytes() {
    return 2u * kKeys * D * 2;  // K then V
}
template <int D>
constexpr uint32_t smem_bytes() {
    return kWarps * kStages * stage_bytes<D>();
}

// CTAs that share W units: no more than there are units
__device__ __forceinline__ int sharers(int64_t W, int ctas) { return W < ctas ? static_cast<int>(W) : ctas; }
// The share of CTA c of n: [W c / n, W (c + 1) / n), never empty
__device__ __forceinline__ int64_t share(int64_t W, int c, int n) { return W * c / n; }

template <int D>
__global__ void __launch_bounds__(kThreads, 2) paged_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int kChunks = D / 8;  // 16-byte chunks a row
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t sums[2 * kWarps];
    __shared__ int64_t found[2];  // sequence and units in front of it
    __shared__ int any_bad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_seq = a.c.heads_kv * a.chunks;  // (key head, head chunk) pairs
    if (threadIdx.x == 0) any_bad = 0;
    bool bad = false;

    allow_dependents();  // the join starts beside this launch, up to its wait
    // this CTA's run of units
    const int first_len = threadIdx.x < a.c.seqs ? clean_len(a, threadIdx.x, &bad) : 0;
    int64_t tiles = 0;
    {
        for (int i = threadIdx.x; i < a.c.seqs; i += kThreads)
            tiles += tiles_of(i == threadIdx.x ? first_len : clean_len(a, i, &bad));
#pragma unroll
        for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        if (lane == 0) sums[kWarps + warp] = tiles;
        __syncthreads();
        tiles = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) tiles += sums[kWarps + w];
    }
    const int64_t W = tiles * per_seq;
    const int n_share = sharers(W, gridDim.x);
    const bool mine = static_cast<int>(blockIdx.x) < n_share;
    const int64_t u0 = mine ? share(W, blockIdx.x, n_share) : 0, u1 = mine ? share(W, blockIdx.x + 1, n_share) : 0;
    if (u0 < u1) {
        // the sequence of unit u0: scans of kThreads sequences at a time
        int64_t carry = 0;
        for (int base = 0; base < a.c.seqs; base += kThreads) {
            const int s = base + threadIdx.x;
            const int len = base == 0 ? first_len : s < a.c.seqs ? clean_len(a, s, &bad) : 0;
            const int64_t n = static_cast<int64_t>(tiles_of(len)) * per_seq;
            int64_t incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            if (base > 0) __syncthreads();
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
            int64_t front = carry;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) front += sums[w];
                carry += sums[w];
            }
            const int64_t before = front + incl - n;
            if (u0 >= before && u0 < before + n) {
                found[0] = s;
                found[1] = before;
            }
            if (carry > u0) break;  // uniform: carry is the same in all threads
        }
        __syncthreads();
        int s = static_cast<int>(found[0]);
        int64_t seq_u = found[1];  // first unit of sequence s

        const uint32_t ring = smem_addr(smem) + warp * kStages * stage_bytes<D>();
        for (int64_t u = u0; u < u1;) {
            int len = clean_len(a, s, &bad);
            int nt = tiles_of(len);
            while (u >= seq_u + static_cast<int64_t>(nt) * per_seq) {  // next sequence (skips empty ones)
                seq_u += static_cast<int64_t>(nt) * per_seq;
                ++s;
                len = clean_len(a, s, &bad);
                nt = tiles_of(len);
            }
            const int pair = static_cast<int>((u - seq_u) / nt);
            const int64_t pair_u = seq_u + static_cast<int64_t>(pair) * nt;
            const int tile0 = static_cast<int>(u - pair_u);
            const int64_t stop = pair_u + nt < u1 ? pair_u + nt : u1;
            const int tile1 = static_cast<int>(stop - pair_u);
            const int hk = pair / a.chunks, hc = pair % a.chunks;
            const int nh = min(kPagedHeads, a.group - hc * kPagedHeads);  // heads of this chunk
            const int h0 = hk * a.group + hc * kPagedHeads;

            // Q: A operand of m16n8k16, rows = heads
            uint32_t qa[D / 16][4];
            {
                const int r = lane >> 2, col = 2 * (lane & 3);
                const __nv_bfloat16 *q = a.q + s * a.q_token + h0 * a.q_head;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = r + 8 * (e & 1), cc = 16 * kk + col + 8 * (e >> 1);
                        qa[kk][e] = row < nh ? __ldg(reinterpret_cast<const uint32_t *>(q + row * a.q_head + cc)) : 0u;
                    }
            }
            const int steps = tile1 - tile0;
            const int32_t *tab = a.c.table + static_cast<int64_t>(s) * a.c.width;
            const int64_t ko = hk * a.c.k_head, vo = hk * a.c.v_head;
            // page of this lane's key (lanes 0-15; the others repeat them) of a step
            auto key_of = [&](int i) { return (tile0 + i) * kTileKeys + warp * kKeys + (lane & 15); };
            auto page_of = [&](int i) -> int {
                const int p = key_of(i);
                return i < steps && p < len ? __ldg(tab + p / a.c.page_size) : 0;
            };
            uint32_t live_of[kStages];  // bit k: key k of the stage counts
            auto fetch = [&](int i, int page, int slot) {
                if (i < steps) {
                    const int p = key_of(i);
                    const bool in = p < len;
                    const bool ok = in && page >= 0 && page < a.c.pages;
                    bad |= in && !ok;
                    const int64_t r = p % a.c.page_size;
                    const int64_t kp = ok ? page * a.c.k_page + r * a.c.k_token + ko : 0;
                    const int64_t vp = ok ? page * a.c.v_page + r * a.c.v_token + vo : 0;
                    const uint32_t live = __ballot_sync(0xffffffffu, ok) & 0xffffu;
#pragma unroll
                    for (int q = 0; q < kStages; ++q)
                        if (q == slot) live_of[q] = live;
                    const uint32_t sk = ring + slot * stage_bytes<D>(), sv = sk + kKeys * D * 2;
#pragma unroll
                    for (int x = 0; x < kKeys * kChunks / 32; ++x) {
                        const int key = (x * 32 + lane) / kChunks, c = lane % kChunks;
                        const int64_t kr = __shfl_sync(0xffffffffu, kp, key);
                        const int64_t vr = __shfl_sync(0xffffffffu, vp, key);
                        const bool take = (live >> key) & 1u;
                        cp_async16_or_zero(sk + swz<kChunks>(key, c), a.c.k + kr + 8 * c, take);
                        cp_async16_or_zero(sv + swz<kChunks>(key, c), a.c.v + vr + 8 * c, take);
                    }
                }
                cp_async_commit();
            };

            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // rows lane/4 and + 8
            float acc[D / 8][4];
#pragma unroll
            for (int n = 0; n < D / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) fetch(i, page_of(i), i);
            int page = page_of(kStages - 1);
            for (int i = 0; i < steps; ++i) {
                const int slot = i % kStages;
                // the slot of step i - 1 is free: this warp has read it
                fetch(i + kStages - 1, page, (i + kStages - 1) % kStages);
                page = page_of(i + kStages);
                cp_async_wait<kStages - 1>();
                __syncwarp();
                uint32_t live = 0;
#pragma unroll
                for (int q = 0; q < kStages; ++q)
                    if (q == slot) live = live_of[q];
                if (live == 0) continue;  // uniform
                const uint32_t sk = ring + slot * stage_bytes<D>(), sv = sk + kKeys * D * 2;
                float sc[2][4] = {};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    // keys 0-7 and 8-15 x 16 features: B operands of two n-tiles
                    uint32_t b0, b1, b2, b3;
                    const int key = (lane & 7) + ((lane >> 4) << 3), c = 2 * kk + ((lane >> 3) & 1);
                    ldsm_x4(sk + swz<kChunks>(key, c), b0, b1, b2, b3);
                    mma_bf16(sc[0], qa[kk], b0, b1);
                    mma_bf16(sc[1], qa[kk], b2, b3);
                }
                if (live != 0xffffu) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!((live >> (8 * n + 2 * (lane & 3) + (e & 1))) & 1u)) sc[n][e] = -INFINITY;
                }
                float mn[2], al[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    mn[h] = fmaxf(m[h], x * a.c2);
                }
                if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        al[h] = m[h] == -INFINITY ? 0.f : fast_exp2(m[h] - mn[h]);
                        l[h] *= al[h];
                        m[h] = mn[h];
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        acc[n][0] *= al[0];
                        acc[n][1] *= al[0];
                        acc[n][2] *= al[1];
                        acc[n][3] *= al[1];
                    }
                }
                uint32_t pa[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ref = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float p0 = fast_exp2(fmaf(sc[n][2 * h], a.c2, -ref));
                        const float p1 = fast_exp2(fmaf(sc[n][2 * h + 1], a.c2, -ref));
                        l[h] += p0 + p1;
                        pa[h + 2 * n] = pack_bf16(p0, p1);
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    // 16 keys x 16 features of V, transposed: B operands of two n-tiles
                    uint32_t b0, b1, b2, b3;
                    const int key = (lane & 7) + (((lane >> 3) & 1) << 3), c = 2 * n + (lane >> 4);
                    ldsm_x4_t(sv + swz<kChunks>(key, c), b0, b1, b2, b3);
                    mma_bf16(acc[2 * n], pa, b0, b1);
                    mma_bf16(acc[2 * n + 1], pa, b2, b3);
                }
            }
            cp_async_wait<0>();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            }
            // join the warps: (m, l) and o of each through shared memory (the rings are idle)
            __syncthreads();
            float *so = reinterpret_cast<float *>(smem);  // [warp][16][D]
            float *sml = so + kWarps * kPagedHeads * D;   // [warp][16][2]
            {
                const int r = lane >> 2, col = 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    float *p = so + (warp * kPagedHeads + r) * D + 8 * n + col;
                    *reinterpret_cast<float2 *>(p) = make_float2(acc[n][0], acc[n][1]);
                    *reinterpret_cast<float2 *>(p + 8 * D) = make_float2(acc[n][2], acc[n][3]);
                }
                if ((lane & 3) == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        sml[(warp * kPagedHeads + r + 8 * h) * 2] = m[h];
                        sml[(warp * kPagedHeads + r + 8 * h) * 2 + 1] = l[h];
                    }
                }
            }
            __syncthreads();
            const bool whole = tile0 == 0 && tile1 == nt;
            // a piece whose (sequence, head) began in an earlier CTA: slot 0, else slot 1
            const int slot = 2 * blockIdx.x + (tile0 == 0 ? 1 : 0);
            for (int x = threadIdx.x; x < nh * (D / 4); x += kThreads) {
                const int r = x / (D / 4), c = 4 * (x % (D / 4));
                float mm = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sml[(w * kPagedHeads + r) * 2]);
                const float ref = mm == -INFINITY ? 0.f : mm;
                float ll = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float sw = fast_exp2(sml[(w * kPagedHeads + r) * 2] - ref);
                    ll += sw * sml[(w * kPagedHeads + r) * 2 + 1];
                    const float4 v = *reinterpret_cast<const float4 *>(so + (w * kPagedHeads + r) * D + c);
                    o.x += sw * v.x;
                    o.y += sw * v.y;
                    o.z += sw * v.z;
                    o.w += sw * v.w;
                }
                if (whole) {
                    const float inv = ll == 0.f ? 0.f : 1.f / ll;
                    uint2 w;
                    w.x = pack_bf16(o.x * inv, o.y * inv);
                    w.y = pack_bf16(o.z * inv, o.w * inv);
                    *reinterpret_cast<uint2 *>(a.o + s * a.o_token + (h0 + r) * a.o_head + c) = w;
                    if (c == 0 && a.lse != nullptr)
                        a.lse[static_cast<int64_t>(s) * a.heads + h0 + r] =
                            ll > 0.f ? (mm + log2f(ll)) * kLn2 : ll == 0.f ? -INFINITY : ll;
                } else {
                    *reinterpret_cast<float4 *>(a.part + (static_cast<int64_t>(slot) * kPagedHeads + r) * D + c) = o;
                    if (c == 0) {
                        float *ml = a.part + static_cast<int64_t>(2 * a.ctas) * kPagedHeads * D +
                                    (slot * kPagedHeads + r) * 2;
                        ml[0] = mm;
                        ml[1] = ll;
                    }
                }
            }
            __syncthreads();  // the rings are refilled next
            u = stop;
        }
    }
    if (bad) any_bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) a.flags[blockIdx.x] = any_bad;
}

// One CTA per (sequence, query head), or with kRange one for a run of them: adds the
// pieces of the CTAs that shared it, in order, its NW warps taking every NW-th
// piece; writes empty rows; the first CTA gathers the flags into the status word.
template <int D, int NW, bool kRange>
__global__ void __launch_bounds__(32 * NW) join_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int kPer = D / 32, NT = 32 * NW;
    __shared__ int64_t sums[2 * NW];
    __shared__ float so[NW][D], sw[kPagedCtas], part[2][NW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(a.c.seqs) * a.heads;
    const int64_t row0 = kRange ? rows * blockIdx.x / gridDim.x : blockIdx.x;
    int s = static_cast<int>(row0 / a.heads), head = static_cast<int>(row0 % a.heads);
    int64_t front, tiles;
    tile_sums<NT>(a, s, sums, &front, &tiles);
    bool bad = false;
    int nt = tiles_of(clean_len(a, s, &bad));
    const int per_seq = a.c.heads_kv * a.chunks;
    const int64_t W = tiles * per_seq;
    const int n = sharers(W, a.ctas);
    auto wait = [&]() {
        wait_for_prerequisites();
        if (blockIdx.x == 0) {
            for (int i = threadIdx.x; i < a.c.seqs; i += NT) clean_len(a, i, &bad);
            for (int i = threadIdx.x; i < a.ctas; i += NT) bad |= a.flags[i] != 0;
            bad = __syncthreads_or(bad);
            if (threadIdx.x == 0) *a.status = bad ? kDevParam : kDevOk;
        }
    };
    auto join = [&]() {
        const int hk = head / a.group, g = head % a.group;
        const int pair = hk * a.chunks + g / kPagedHeads, r = g % kPagedHeads;
        const int64_t first = front * per_seq + static_cast<int64_t>(pair) * nt;
        // the CTA of unit u is the last one whose share begins at or before it
        int c0 = 0, c1 = 0;
        if (nt > 0) {
            c0 = static_cast<int>(((first + 1) * n - 1) / W);
            c1 = static_cast<int>(((first + nt) * n - 1) / W);
        }
        if constexpr (!kRange) wait();
        __nv_bfloat16 *dst = a.o + s * a.o_token + head * a.o_head;
        float *lse = a.lse == nullptr ? nullptr : a.lse + static_cast<int64_t>(s) * a.heads + head;
        if (nt == 0) {
            for (int d = threadIdx.x; d < D; d += NT) dst[d] = __float2bfloat16_rn(0.f);
            if (threadIdx.x == 0 && lse != nullptr) *lse = -INFINITY;
            return;
        }
        if (c0 == c1) return;  // written whole
        const int pieces = c1 - c0 + 1;
        const float2 *ml = reinterpret_cast<const float2 *>(a.part + static_cast<int64_t>(2 * a.ctas) * kPagedHeads * D);
        // piece p: the first one began in its CTA (slot 1), the others in an earlier one (slot 0)
        auto slot_of = [&](int p) { return static_cast<int64_t>(2 * (c0 + p) + (p == 0 ? 1 : 0)) * kPagedHeads + r; };
        float m[(kPagedCtas + NT - 1) / NT], l[(kPagedCtas + NT - 1) / NT], M = -INFINITY;
#pragma unroll
        for (int i = 0; i < (kPagedCtas + NT - 1) / NT; ++i) {
            const int p = i * NT + threadIdx.x;
            m[i] = -INFINITY;
            l[i] = 0.f;
            if (p < pieces) {
                const float2 v = ml[slot_of(p)];
                m[i] = v.x;
                l[i] = v.y;
            }
            M = fmaxf(M, m[i]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (lane == 0) part[0][warp] = M;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, part[0][w]);
        const float R = M == -INFINITY ? 0.f : M;
        float total = 0.f;
#pragma unroll
        for (int i = 0; i < (kPagedCtas + NT - 1) / NT; ++i) {
            const int p = i * NT + threadIdx.x;
            const float w = fast_exp2(m[i] - R);
            if (p < pieces) sw[p] = w;
            total += w * l[i];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (lane == 0) part[1][warp] = total;
        __syncthreads();
        total = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) total += part[1][w];
        float o[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = 0.f;
#pragma unroll 8
        for (int p = warp; p < pieces; p += NW) {
            const float *src = a.part + slot_of(p) * D + lane * kPer;
            const float w = sw[p];
            if constexpr (kPer == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src);
                o[0] += w * v.x;
                o[1] += w * v.y;
                o[2] += w * v.z;
                o[3] += w * v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(src);
                o[0] += w * v.x;
                o[1] += w * v.y;
            }
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = o[e];
        __syncthreads();
        const float inv = total == 0.f ? 0.f : 1.f / total;
        for (int d = threadIdx.x; d < D; d += NT) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) x += so[w][d];
            dst[d] = __float2bfloat16_rn(x * inv);
        }
        if (threadIdx.x == 0 && lse != nullptr)
            *lse = total > 0.f ? (M + log2f(total)) * kLn2 : total == 0.f ? -INFINITY : total;
    };
    if constexpr (!kRange) {
        join();
    } else {
        wait();
        const int64_t count = rows * (blockIdx.x + 1) / gridDim.x - row0;
        for (int64_t i = 0; i < count; ++i) {
            if (i > 0) {
                __syncthreads();  // the row before has been read from shared memory
                if (++head == a.heads) {
                    head = 0;
                    front += nt;
                    nt = tiles_of(clean_len(a, ++s, &bad));
                }
            }
            join();
        }
    }
}

}  // namespace paged
}  // namespace nabla

cudaError_t nabla_launch_append(const nabla::AppendArgs &a, cudaStream_t stream) {
    // up to 8 tokens a CTA (4 took 37 us where 8 take 33, at 134 MB); fewer until
    // the GPU is full (four CTAs an SM)
    int64_t per = a.total / (4 * 148);
    per = per < 1 ? 1 : per > nabla::paged::kAppendTokens ? nabla::paged::kAppendTokens : per;
    int64_t blocks = (a.total + per - 1) / per;
    // every CTA looks at every border: with many of them no more CTAs than run at once,
    // or that work grows with their square (sequences of 20 rows: 1,500 31 us either way,
    // 3,000 53 against 57, 20,000 320 against 760)
    const bool stride = a.cu != nullptr && a.c.seqs > 1024 && blocks > 8 * 148;
    if (stride) blocks = 8 * 148;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (stride)
        nabla::paged::append_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a, static_cast<int>(per));
    else
        nabla::paged::append_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a, static_cast<int>(per));
    return cudaGetLastError();
}

constexpr int kFewSeqs = 256;
constexpr unsigned kJoinCtas = 16 * 148;  // of 128 threads, what runs at once

template <int D>
static cudaError_t launch_paged(const nabla::PagedArgs &a, cudaStream_t stream) {
    using namespace nabla::paged;
    cudaError_t err = nabla_allow_smem<paged_kernel<D>>(smem_bytes<D>());
    if (err != cudaSuccess) return err;
    paged_kernel<D><<<a.ctas, kThreads, smem_bytes<D>(), stream>>>(a);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    // few rows to join may each have hundreds of pieces: 16 warps a row (100,000
    // keys, 8 heads on one key head: 22 us against 37 with 4); many rows have a few
    // pieces each, which four warps add while other rows have theirs
    // Every CTA looks at all lengths: with many sequences no more CTAs than run at once, or
    // that work grows with their square (the whole call, up to 1,000 rows and 40 heads each:
    // 256 sequences 152 us against 150 with a CTA a row, 512 254 against 260, 1,000 451 against
    // 481; 6,000 of 20 rows and 8 heads 229 against 424)
    const unsigned rows = static_cast<unsigned>(a.c.seqs * a.heads);
    if (rows <= 148) return nabla_launch_early(join_kernel<D, 16, false>, rows, 512, 0, stream, a);
    if (a.c.seqs <= kFewSeqs || rows <= kJoinCtas)
        return nabla_launch_early(join_kernel<D, 4, false>, rows, 128, 0, stream, a);
    return nabla_launch_early(join_kernel<D, 4, true>, kJoinCtas, 128, 0, stream, a);
}

cudaError_t nabla_launch_paged(const nabla::PagedArgs &a, cudaStream_t stream) {
    return a.c.D == 128 ? launch_paged<128>(a, stream) : launch_paged<64>(a, stream);
}
