// Attention of packed sequences, backward, on tcgen05 tensor cores (D = 128 or
// 64), deterministic: every output row has one writer, no atomics.
//   delta_i = dout_i . o_i,  P = exp(scale q.k - lse),  dS = P (dout.v - delta),
//   dV = P^T dout,  dK = scale dS^T Q,  dQ = scale dS K.
//
// pre_kernel: delta and lse log2(e) (both negated, the form the exponent and the
//   difference take) into arrays in which every sequence starts at a multiple
//   of 64 rows, so that a tile's 64 values are one aligned bulk copy; rows
//   that pad a sequence, and rows that keep no key, hold -inf: their P is 0.
// dkdv_kernel: one CTA per 128 keys of a sequence and key head, walking the
//   query heads of the group and their tiles of 64 queries:
//     S^T = K Q^T (K a TMEM operand), dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   so the gradients of shared heads add up in TMEM, in a fixed order.
// dq_kernel: one CTA per 128 rows (token, head of the group; as the forward),
//   walking tiles of 64 keys:
//     S = Q K^T, dP = dO V^T (Q, dO TMEM operands), dQ += dS K
//
// Seven products per pair against the five that one kernel with atomic sums of
// dQ would need: the price of sums whose order does not change.  P and dS are
// rounded to bf16 for their MMAs (by up to 2^-8 relative each), everything else is
// float32.  MMAs go out four per elect.sync from converged warps (an N = 64 MMA
// is accepted about when it starts, so the issuer must not fall behind).
//
// delta = dout . o takes o as it was rounded to bf16.  With many keys that is small
// against the rounding of dS; with few, dP - delta cancels and the rounding of o
// stays: over sequences of 3 rows the gradients were off by 0.5%, of 2 rows by 3%.
// So for every row that keeps at most 64 keys -- all of them in the first tile of its
// sequence, whatever else the row's tile or unit holds -- delta is the sum over
// that tile of P dP in float32, the same number unrounded.  (Taking o again from q, k
// and v in pre_kernel instead cost 96 us for 4,096 rows and 24 heads on 30 keys.)
//
// Rows behind a sequence inside a tile: scores are replaced by -inf, and rows
// that are summed over (Q and dO in dkdv, K in dq) are zeroed in shared memory,
// as 0 * NaN would spread.  Waits are bounded as in the forward.
#include <type_traits>

#include "packed.cuh"

namespace nabla {
namespace packed {

using namespace sm100;

constexpr uint32_t kHalfTile = 16384;  // 128 rows x 64 features bf16
constexpr int kPreThreads = 256;

// ---------------------------------------------------------------------------
// delta and lse, padded: one CTA per 64 rows of a sequence and `per` heads
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(kPreThreads) pre_kernel(const __grid_constant__ Args a, int per) {
    __shared__ SeqTile st;
    allow_dependents();
    // the borders, shared out over the launch (there are no fewer CTAs in x than sequences)
    if (blockIdx.y == 0 && !borders_ok(a, static_cast<int64_t>(blockIdx.x) * kPreThreads + threadIdx.x, 1 << 30)) {
        atomicExch(a.status, kDevParam);
        atomicExch(a.status + 2, 1);
    }
    if (!find_seq(a, true, 64, blockIdx.x, &st)) return;
    constexpr int TPR = D / 8;  // threads per row, 8 features each
    constexpr int kStep = kPreThreads / TPR;
    const int sub = threadIdx.x % TPR;
    const int h1 = min(a.heads, static_cast<int>(blockIdx.y + 1) * per);
    for (int h = blockIdx.y * per; h < h1; ++h) {
        const int64_t base = h * a.pad_rows + static_cast<int64_t>(st.pad + st.tile) * 64;
#pragma unroll
        for (int r = threadIdx.x / TPR; r < 64; r += kStep) {
            const int i = st.tile * 64 + r;
            float acc = 0.f;
            if (i < st.Lq) {
                const int64_t tok = st.q0 + i;
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(a.o.row(tok, h)) + sub);
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(a.dout.row(tok, h)) + sub);
                const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&u);
                const __nv_bfloat162 *y = reinterpret_cast<const __nv_bfloat162 *>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p = __bfloat1622float2(x[e]), q = __bfloat1622float2(y[e]);
                    acc = fmaf(p.x, q.x, acc);
                    acc = fmaf(p.y, q.y, acc);
                }
            }
#pragma unroll
            for (int o = 1; o < TPR; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (sub == 0) {
                const float L = i < st.Lq ? a.lse[h * a.total_q + st.q0 + i] : -INFINITY;
                a.pad_d[base + r] = L == -INFINITY ? 0.f : -acc;
                a.pad_l[base + r] = L == -INFINITY ? -INFINITY : -(L * 1.4426950408889634f);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
constexpr int kStages = 4;
constexpr int kKvThreads = 320;
template <int D>
struct KvLayout {
    static constexpr int kHalves = D / 64;
    static constexpr uint32_t kQBytes = 64u * D * 2;  // 64 queries
    static constexpr uint32_t kStageBytes = ((2 * kQBytes + 512 + 1023) / 1024) * 1024;
    static constexpr uint32_t KV_V = 0;
    static constexpr uint32_t KV_RING = kHalves * kHalfTile;
    static constexpr uint32_t KV_BAR = KV_RING + kStages * kStageBytes;
    static constexpr int kBars = 1 + 2 * kStages + 2 + 2 + 1 + 1 + 1 + 1;
    static constexpr uint32_t KV_COL = (KV_BAR + 8 * kBars + 15) / 16 * 16;  // sums over keys: [2][2][64]
    static constexpr uint32_t KV_SEQ = KV_COL + 2 * 2 * 64 * 4;
    static constexpr uint32_t KV_INT = (KV_SEQ + sizeof(SeqTile) + 7) / 8 * 8;
    static constexpr uint32_t kSmem = KV_INT + 16 + 1024;
};

// TMEM columns: S^T(t) [64 (t&1), +64), dP^T [128, 192), K [192, 192 + D/2),
// dV [256, 256 + D), dK [384, 384 + D).  Warpgroup qg handles queries
// [32 qg, +32) of the tile and writes bf16 P^T and dS^T over its own S^T
// columns, P^T at [32 qg, +16) and dS^T at [32 qg + 16, +16).
constexpr uint32_t kColDP = 128, kColK = 192;
template <int D>
__global__ void __launch_bounds__(kKvThreads, 1)
    dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tv,
                const __grid_constant__ CUtensorMap tdo, const __grid_constant__ Args a) {
    using L = KvLayout<D>;
    constexpr int kHalves = L::kHalves;
    constexpr uint32_t kQBytes = L::kQBytes, kStageBytes = L::kStageBytes;
    constexpr uint32_t KV_V = L::KV_V, KV_RING = L::KV_RING;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    unsigned char *sm = smem_raw + pad;
    const uint32_t sb = raw + pad;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::KV_BAR);
    uint64_t *kv_full = bar, *st_full = bar + 1, *st_empty = bar + 1 + kStages;
    // pd_full[t & 1]: the eight softmax warps wrote P^T(t), dS^T(t)
    uint64_t *s_full = bar + 1 + 2 * kStages, *pd_full = s_full + 2, *done = pd_full + 2;
    // k_ready: K is in TMEM; dp_free: the dP^T of the current tile is in
    // registers; raw_full: a stage that still has rows to zero has arrived
    uint64_t *k_ready = done + 1, *dp_free = k_ready + 1, *raw_full = dp_free + 1;
    SeqTile *st = reinterpret_cast<SeqTile *>(sm + L::KV_SEQ);
    int *sInt = reinterpret_cast<int *>(sm + L::KV_INT);
    volatile int *abort_flag = sInt + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = static_cast<int>(blockIdx.x % a.heads_kv);
    if (!find_seq(a, false, 128, blockIdx.x / a.heads_kv, st)) {
        // (an exit counts as both of the calls below; behind the wait, so that dQ, and with it
        // the end of the call, never comes in front of the end of pre_kernel)
        wait_for_prerequisites();
        return;
    }
    const int Lq = st->Lq, Lk = st->Lk, off = Lk - Lq, G = a.group;
    const int j0 = st->tile * 128;  // first key
    // query tiles [qs, qs + per) of each head: query i keeps keys up to i + off
    const int qs = a.causal ? max(0, j0 - off) >> 6 : 0;
    const int per = max(0, ((Lq + 63) >> 6) - qs);

    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&st_full[s], 1);
            mbar_init(&st_empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&pd_full[b], 8);
        }
        mbar_init(done, 1);
        mbar_init(k_ready, 8);
        mbar_init(dp_free, 8);
        mbar_init(raw_full, 1);
        sInt[2] = sInt[3] = *reinterpret_cast<volatile int *>(a.status) != 0 ? 1 : 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(&sInt[0]), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(sInt[0]);
    const int ntiles = G * per;
    // pre_kernel has finished from here on; then dQ's CTAs may take the SMs that
    // this launch leaves idle (they read nothing that it writes)
    wait_for_prerequisites();
    allow_dependents();
    const bool bad = *reinterpret_cast<volatile int *>(a.status + 2) != 0;  // (read for the stores at the end)

    if (warp == 0) {
        // ---------------- producer: V once, then the query stages ----------------
        int t = 0, tails = 0;
        if (ntiles > 0) {
            if (lane == 0) {
                prefetch_tmap(&tq);
                prefetch_tmap(&tdo);
                mbar_expect_tx(kv_full, kHalves * kHalfTile);
                for (int h = 0; h < kHalves; ++h)
                    tma_load_3d(sb + KV_V + h * kHalfTile, &tv, kv_full, 64 * h, hk, st->k0 + j0);
            }
            for (; t < ntiles && !a.stall; ++t) {
                const int s = t % kStages, g = t / per, i0 = (qs + t % per) * 64;
                const bool ok = __all_sync(
                    0xffffffffu, lane != 0 || wait_bar(&st_empty[s], ((t / kStages) & 1) ^ 1,
                                                       abort_flag, a.status, a.limit));
                if (!ok) break;
                const uint32_t dst = sb + KV_RING + s * kStageBytes;
                const int live = Lq - i0;
                const bool zero = live < 64 && st->q0 + Lq < a.total_q;
                uint64_t *full = zero ? raw_full : &st_full[s];
                if (lane == 0) {
                    const int hq = hk * G + g;
                    mbar_expect_tx(full, 2 * kQBytes + 512);
                    for (int h = 0; h < kHalves; ++h) {  // [Q halves][dO halves], 8 KB each
                        tma_load_3d(dst + h * 8192, &tq, full, 64 * h, hq, st->q0 + i0);
                        tma_load_3d(dst + kQBytes + h * 8192, &tdo, full, 64 * h, hq, st->q0 + i0);
                    }
                    const int64_t y = hq * a.pad_rows + static_cast<int64_t>(st->pad) * 64 + i0;
                    bulk_load(dst + 2 * kQBytes, a.pad_l + y, 256, full);
                    bulk_load(dst + 2 * kQBytes + 256, a.pad_d + y, 256, full);
                }
                __syncwarp();
                if (zero) {  // the last tile of each head
                    const bool in = wait_plain(raw_full, tails++ & 1, a.limit);
                    if (!__all_sync(0xffffffffu, in)) break;
                    zero_rows(sm + KV_RING + s * kStageBytes, live, 64, 2 * kHalves, 8192, lane);
                    if (lane == 0) mbar_arrive(&st_full[s]);
                }
            }
            // drain: never leave with a copy in flight
            if (lane == 0) {
                wait_plain(kv_full, 0, a.limit);
                for (int u = t > kStages ? t - kStages : 0; u < t; ++u)
                    wait_plain(&st_full[u % kStages], (u / kStages) & 1, a.limit);
            }
        }
    } else if (warp == 1) {
        // MMA issuer: whole warp, one elected lane issues
        constexpr uint32_t kIdS = idesc_bf16(128, 64, 0, 0);    // K . Q^T, V . dO^T
        constexpr uint32_t kIdG = idesc_bf16(128, D, 0, 1);     // P^T . dO, dS^T . Q
        // Shared-memory descriptors advance by (byte offset >> 4) in their low
        // 14-bit address field; every tile address here stays below 2^18.
        const uint64_t dV = desc_sw128(sb + KV_V, 16, 1024);
        auto SdP = [&](int t) -> bool {
            const int s = t % kStages;
            if (!warp_wait(&st_full[s], (t / kStages) & 1, abort_flag, a.status, a.limit))
                return false;
            tc_fence_after();
            const uint32_t st = sb + KV_RING + s * kStageBytes;
            const uint64_t dQ = desc_sw128(st, 16, 1024), dO = desc_sw128(st + kQBytes, 16, 1024);
            const uint32_t s0 = tmem + (t & 1) * 64, p0 = tmem + kColDP;
            // byte offsets of k-step kk (16 features) in a K-major tile of one
            // key / query block pair: 64-feature halves kHalfTile / 8192 apart
            auto offA = [](int kk) {
                return static_cast<uint32_t>(((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4);
            };
            auto offB = [](int kk) {
                return static_cast<uint32_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4);
            };
            // S^T first (K from TMEM, Q from shared memory) ...
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 4)
                mma_ts4_warp(s0, s0, s0, s0, tmem + kColK + 8 * kk, tmem + kColK + 8 * kk + 8,
                             tmem + kColK + 8 * kk + 16, tmem + kColK + 8 * kk + 24, dQ + offB(kk),
                             dQ + offB(kk + 1), dQ + offB(kk + 2), dQ + offB(kk + 3), kIdS, kk > 0, 1u);
            // ... then dP^T into the single buffer, once the softmax warps hold
            // tile t - 1's in registers
            if (t > 0 && !warp_wait(dp_free, (t - 1) & 1, abort_flag, a.status, a.limit))
                return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; kk += 4)
                mma_ss4_warp(p0, p0, p0, p0, dV + offA(kk), dV + offA(kk + 1), dV + offA(kk + 2),
                             dV + offA(kk + 3), dO + offB(kk), dO + offB(kk + 1), dO + offB(kk + 2),
                             dO + offB(kk + 3), kIdS, kk > 0, 1u);
            mma_commit_warp(&s_full[t & 1]);
            return true;
        };
        auto Grad = [&](int t) -> bool {
            const int s = t % kStages;
            if (!warp_wait(&pd_full[t & 1], (t >> 1) & 1, abort_flag, a.status, a.limit))
                return false;
            tc_fence_after();
            const uint32_t st = sb + KV_RING + s * kStageBytes;
            // dO, Q as MN-major B operands; query k-step kk (16 queries) starts
            // 2048 bytes further and reads bf16 P^T / dS^T columns
            // 32 (kk / 2) + 8 (kk % 2) / + 16 of this tile's S^T buffer
            const uint64_t gO = desc_sw128(st + kQBytes, 8192, 1024), gQ = desc_sw128(st, 8192, 1024);
            const uint32_t c = tmem + (t & 1) * 64;
            const uint32_t f = t > 0 ? 1u : 0u;
            mma_ts4_warp(tmem + 256, tmem + 384, tmem + 256, tmem + 384, c, c + 16, c + 8, c + 24,
                         gO, gQ, gO + 128, gQ + 128, kIdG, f, f);
            mma_ts4_warp(tmem + 256, tmem + 384, tmem + 256, tmem + 384, c + 32, c + 48, c + 40,
                         c + 56, gO + 256, gQ + 256, gO + 384, gQ + 384, kIdG, 1u, 1u);
            mma_commit_warp(&st_empty[s]);
            return true;
        };
        if (ntiles > 0 && warp_wait(kv_full, 0, abort_flag, a.status, a.limit) &&
            warp_wait(k_ready, 0, abort_flag, a.status, a.limit)) {
            bool ok = SdP(0);
            for (int t = 0; ok && t < ntiles; ++t) {
                if (t + 1 < ntiles) ok = SdP(t + 1);
                ok = ok && Grad(t);
            }
        }
        mma_commit_warp(done);
        if (lane == 0) wait_plain(done, 0, a.limit);
        __syncwarp();
    } else {
        const int wq = warp & 3;
        const int qg = (warp - 2) >> 2;  // queries [32 qg, 32 qg + 32) of each tile
        const int tw = wq * 32 + lane;   // key row 0..127
        const int key = j0 + tw;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        bool ok = true;
        {
            // features [D/2 qg, D/2 qg + D/2) of the key's row -> TMEM columns
            // [kColK + D/4 qg, +D/4); keys behind the sequence are zero
            uint32_t kv[D / 4];
            const uint4 *src = reinterpret_cast<const uint4 *>(a.k.row(st->k0 + min(key, Lk - 1), hk) + (D / 2) * qg);
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                const uint4 v = key < Lk ? __ldg(src + e) : make_uint4(0, 0, 0, 0);
                kv[4 * e] = v.x;
                kv[4 * e + 1] = v.y;
                kv[4 * e + 2] = v.z;
                kv[4 * e + 3] = v.w;
            }
            if constexpr (D == 128)
                tmem_st32(tmem + lane_base + kColK + 32 * qg, reinterpret_cast<float *>(kv));
            else
                tmem_st16(tmem + lane_base + kColK + 16 * qg, kv);
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_ready);
        const float c = a.c;
        const uint64_t c2 = f2_pack(c, c);
        // (sInt[3] does not change, unlike the abort flag: the warps that meet at the
        // barriers of a tile below agree on their number)
        const int nt = sInt[3] != 0 ? 0 : ntiles;
        float *col = reinterpret_cast<float *>(sm + L::KV_COL);
        int qt = qs;  // query tile within its head
        // queries in front of `few_end` keep at most 64 keys, all in this tile
        const int few_end = Lk <= 64 ? Lq : a.causal && j0 == 0 ? max(0, min(Lq, 64 - off)) : 0;
        auto tile = [&](int t, auto few) {
            ok = wait_bar(&s_full[t & 1], (t >> 1) & 1, abort_flag, a.status, a.limit) && ok;
            tc_fence_after();
            const uint32_t scol = tmem + lane_base + (t & 1) * 64 + 32 * qg;
            uint32_t pk[16], dk2[16];  // packed bf16 pairs of P^T and dS^T
            const float4 *L4 = reinterpret_cast<const float4 *>(
                sm + KV_RING + (t % kStages) * kStageBytes + 2 * kQBytes + 128 * qg);
            const float4 *D4 = L4 + 16;  // delta follows lse at +256 bytes
            float sv[32], dp[32];
            tmem_ld32(scol, sv);
            tmem_ld32(tmem + lane_base + kColDP + 32 * qg, dp);
            tmem_wait_ld();
            // dP^T is in registers: the buffer may take the next tile's
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dp_free);
            // queries in front of `first` (of this group's 32) do not keep the key
            const int first = a.causal ? key - off - qt * 64 - 32 * qg : 0;
            if (a.causal && j0 + 127 - off > qt * 64 + 32 * qg) {  // uniform: the tile is masked
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    sv[e] = e >= first ? sv[e] : -INFINITY;
                    if constexpr (few.value) dp[e] = e >= first ? dp[e] : 0.f;
                }
            }
            if constexpr (few.value) {
                // P, then delta as the sum of P dP over the keys: lanes and two warps
                // (the first 64 keys, all that such a query keeps)
#pragma unroll
                for (int q4 = 0; q4 < 8; ++q4) {
                    const float4 l4 = L4[q4];
                    const float la[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) sv[4 * q4 + e] = fast_exp2(fmaf(sv[4 * q4 + e], c, la[e]));
                }
                const int end = few_end - qt * 64 - 32 * qg;  // of this group's 32 queries
                float mine = 0.f;
                if (end > 0) {
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = key < Lk ? sv[e] * dp[e] : 0.f;
                    // 32 values of 32 lanes: lane l ends with the sum of value l
#pragma unroll
                    for (int h = 16; h; h >>= 1) {
                        const bool up = lane & h;
#pragma unroll
                        for (int i = 0; i < h; ++i) {
                            const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + h], h);
                            v[i] = (up ? v[i + h] : v[i]) + other;
                        }
                    }
                    mine = v[0];
                }
                // (two buffers, one barrier a tile: S^T of tile t + 2 is issued behind the
                // arrival on pd_full that ends tile t in every warp)
                float *sum = col + (t & 1) * 128;
                if (wq < 2) {
                    // a query that keeps more takes the delta of pre_kernel
                    if (lane >= end) mine = wq == 0 ? -reinterpret_cast<const float *>(D4)[lane] : 0.f;
                    sum[64 * wq + 32 * qg + lane] = mine;
                }
                bar_sync(1 + qg, 128);
                const float4 *A4 = reinterpret_cast<const float4 *>(sum + 32 * qg);
#pragma unroll
                for (int q4 = 0; q4 < 8; ++q4) {
                    const float4 x = A4[q4], y = A4[q4 + 16];
                    const float d[4] = {x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w};
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int q = 4 * q4 + e;
                        pk[q >> 1] = pack_bf16(sv[q], sv[q + 1]);
                        dk2[q >> 1] = pack_bf16(sv[q] * (dp[q] - d[e]), sv[q + 1] * (dp[q + 1] - d[e + 1]));
                    }
                }
            } else {
#pragma unroll
                for (int q4 = 0; q4 < 8; ++q4) {
                    const float4 l4 = L4[q4], d4 = D4[q4];
                    const float la[4] = {l4.x, l4.y, l4.z, l4.w};
                    const float da[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const int q = 4 * q4 + e;
                        const uint64_t x = f2_fma(f2_pack(sv[q], sv[q + 1]), c2, f2_pack(la[e], la[e + 1]));
                        const float p0 = fast_exp2(f2_lo(x)), p1 = fast_exp2(f2_hi(x));
                        const uint64_t g = f2_mul(f2_pack(p0, p1),
                                                  f2_add(f2_pack(dp[q], dp[q + 1]), f2_pack(da[e], da[e + 1])));
                        pk[2 * q4 + (e >> 1)] = pack_bf16(p0, p1);
                        dk2[2 * q4 + (e >> 1)] = pack_bf16(f2_lo(g), f2_hi(g));
                    }
                }
            }
            tmem_st16(scol, pk);
            tmem_st16(scol + 16, dk2);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pd_full[t & 1]);
            if (++qt == qs + per) qt = qs;
        };
        // Two instances, as only the first key tile of a sequence has such queries: in one
        // loop the test cost 4% of a dense walk.  (So did the same condition written
        // with few_end.)
        if (Lk <= 64 || (a.causal && j0 == 0 && off < 64))
            for (int t = 0; t < nt; ++t) tile(t, std::true_type{});
        else
            for (int t = 0; t < nt; ++t) tile(t, std::false_type{});
        if (ok && nt > 0) ok = wait_bar(done, 0, abort_flag, a.status, a.limit);
        tc_fence_after();
        // warp-uniform flags around the collective TMEM loads
        const bool aborted = __any_sync(0xffffffffu, bad || *abort_flag != 0);
        const bool live = __all_sync(0xffffffffu, ok) && nt > 0;
        if (!aborted) {
            // warpgroup 0 writes the dV row, warpgroup 1 the dK row
            __nv_bfloat16 *dst = (qg ? a.dk : a.dv).row(st->k0 + min(key, Lk - 1), hk);
            const float mul = qg ? a.scale : 1.f;
#pragma unroll
            for (int part = 0; part < D / 32; ++part) {
                float v[32];
                if (live) {
                    tmem_ld32(tmem + lane_base + 256 + 128 * qg + 32 * part, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (key < Lk) {
#pragma unroll
                    for (int e8 = 0; e8 < 4; ++e8) {
                        uint4 w;
                        w.x = pack_bf16(v[8 * e8] * mul, v[8 * e8 + 1] * mul);
                        w.y = pack_bf16(v[8 * e8 + 2] * mul, v[8 * e8 + 3] * mul);
                        w.z = pack_bf16(v[8 * e8 + 4] * mul, v[8 * e8 + 5] * mul);
                        w.w = pack_bf16(v[8 * e8 + 6] * mul, v[8 * e8 + 7] * mul);
                        *reinterpret_cast<uint4 *>(dst + 32 * part + 8 * e8) = w;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
// Thread (g, r) of the two dS warpgroups handles row r and keys [32 g, +32) of
// the tile and writes their bf16 dS over its own S columns [32 g, +16).  Two
// warps issue: warp 1 the S and dP MMAs, warp 10 the dQ MMAs.  S and dP have two
// buffers each, so those of a tile run under the softmax of the one before.
// Persistent: a CTA takes units (128 rows) from a counter; the dS warps fetch
// the next unit's Q and dO rows into registers in front of the last one's
// epilogue, and K and V tiles of the next unit run ahead in the ring.  With
// one CTA a unit, 8 key tiles a unit took 11 us each, most of it start and end.
// TMEM columns: S(t) [64 (t % 2), +64), dP(t) 128 further, dQ [256, 256 + D),
// Q [384, 384 + D/2), dO [448, 448 + D/2).
constexpr int kDqThreads = 352;
constexpr int kDqGradWarp = 10;
constexpr uint32_t kDqColDP = 128, kColDQ = 256, kColQ = 384, kColDO = 448;

// One unit, as the loading warp hands it to the others.
struct DqUnit {
    int valid, hk, q0, Lq, k0, Lk, pad;
    int R0;  // first row
    int nt;  // key tiles
};

template <int D>
struct DqLayout {
    static constexpr int kHalves = D / 64;
    static constexpr int kDqRing = D == 128 ? 6 : 10;
    static constexpr uint32_t kBlockBytes = 64u * D * 2;  // 64 keys of K or V
    static constexpr uint32_t kDqSlot = 2 * kBlockBytes;
    static constexpr uint32_t DQ_STAGE = kDqRing * kDqSlot;  // 2 KB per dS warp
    static constexpr uint32_t DQ_RED = DQ_STAGE + 8 * 2048;  // sums over the keys of a half: [2][128]
    static constexpr uint32_t DQ_BAR = DQ_RED + 2 * 128 * 4;
    static constexpr int kBars = 2 * kDqRing + 2 + 2 + 1 + 1 + 2 + 1 + 1 + 4 + 4;
    static constexpr uint32_t DQ_UNIT = DQ_BAR + 8 * kBars;
    static constexpr uint32_t DQ_INT = (DQ_UNIT + 2 * sizeof(DqUnit) + 15) / 16 * 16;
    static constexpr uint32_t kSmem = DQ_INT + 16 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
              const __grid_constant__ Args a) {
    using L = DqLayout<D>;
    constexpr int kHalves = L::kHalves, kDqRing = L::kDqRing;
    constexpr uint32_t kBlockBytes = L::kBlockBytes, kDqSlot = L::kDqSlot;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    unsigned char *sm = smem_raw + pad;
    const uint32_t sRing = raw + pad;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::DQ_BAR);
    uint64_t *kv_full = bar, *kv_empty = bar + kDqRing, *s_full = bar + 2 * kDqRing;
    // per S buffer: s_full (S, dP complete), ds_full (the eight dS warps wrote
    // dS), s_free (the dQ MMAs have read it)
    uint64_t *ds_full = s_full + 2, *q_ready = ds_full + 2, *done = q_ready + 1;
    uint64_t *s_free = done + 1, *sdp_done = s_free + 2, *raw_full = sdp_done + 1;
    uint64_t *u_full = raw_full + 1, *u_empty = u_full + 2;  // per unit slot; read by ten warps
    uint64_t *pair = u_empty + 2;  // the two dS warps that share rows
    volatile DqUnit *units = reinterpret_cast<DqUnit *>(sm + L::DQ_UNIT);
    int *sInt = reinterpret_cast<int *>(sm + L::DQ_INT);  // [0] tmem base [2] abort
    volatile int *abort_flag = sInt + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group;

    if (threadIdx.x == 0) {
        for (int r = 0; r < kDqRing; ++r) {
            mbar_init(&kv_full[r], 1);
            mbar_init(&kv_empty[r], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&ds_full[b], 8);
            mbar_init(&s_free[b], 1);
        }
        mbar_init(q_ready, 8);
        mbar_init(done, 1);
        mbar_init(sdp_done, 1);
        mbar_init(raw_full, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&u_full[b], 1);
            mbar_init(&u_empty[b], 10);
        }
        for (int w = 0; w < 4; ++w) mbar_init(&pair[w], 2);
        sInt[2] = sInt[3] = *reinterpret_cast<volatile int *>(a.status) != 0 ? 1 : 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(&sInt[0]), 512);
        tmem_relinquish();
    }
    const bool good = borders_ok(a, threadIdx.x, kDqThreads);
    tc_fence_before();
    const bool go = !__syncthreads_or(!good);
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(sInt[0]);
    bool ok = go && sInt[3] == 0;  // (not the abort flag: the same in all threads)

    if (warp == 0) {
        // ---------------- producer: units, then their K and V tiles through the ring ----------------
        if (lane == 0) {
            prefetch_tmap(&tk);
            prefetch_tmap(&tv);
        }
        UnitScan scan;
        uint32_t x = blockIdx.x;
        uint32_t seq = 0, tails = 0;
        for (uint32_t n = 0; ok; ++n) {
            const int us = n & 1;
            DqUnit u = {};
            x = __shfl_sync(0xffffffffu, x, 0);
            const uint32_t now = x;
            if (now < a.units) {
                if (lane == 0) x = take_unit(a);  // the next one, under this one's loads
                SeqTile st;
                const uint32_t hkv = a.heads_kv;
                u.hk = static_cast<int>(now % hkv);
                u.valid = scan.find(a, now / hkv, G, 128, lane, &st);
                if (u.valid) {
                    u.q0 = st.q0;
                    u.Lq = st.Lq;
                    u.k0 = st.k0;
                    u.Lk = st.Lk;
                    u.pad = st.pad;
                    const int rows = u.Lq * G;  // below 2^31: heads * total_q is
                    // the last rows of a causal sequence keep the most keys: they go first
                    u.R0 = ((rows + 127) / 128 - 1 - st.tile) * 128;
                    const int last_tok = min(u.R0 + 127, rows - 1) / G;
                    const int kend = a.causal ? min(u.Lk, last_tok + 1 + u.Lk - u.Lq) : u.Lk;
                    u.nt = kend > 0 ? (kend + 63) >> 6 : 0;
                }
            }
            ok = __all_sync(0xffffffffu, lane != 0 || wait_bar(&u_empty[us], ((n >> 1) & 1u) ^ 1u, abort_flag,
                                                               a.status, a.limit));
            if (!ok) break;
            if (lane == 0) {
                volatile DqUnit &w = units[us];
                w.valid = u.valid;
                w.hk = u.hk;
                w.q0 = u.q0;
                w.Lq = u.Lq;
                w.k0 = u.k0;
                w.Lk = u.Lk;
                w.pad = u.pad;
                w.R0 = u.R0;
                w.nt = u.nt;
                mbar_arrive(&u_full[us]);
            }
            __syncwarp();
            if (!u.valid || a.stall) break;
            for (int t = 0; ok && t < u.nt; ++t) {
                const int slot = seq % kDqRing;
                ok = __all_sync(0xffffffffu, lane != 0 || wait_bar(&kv_empty[slot], ((seq / kDqRing) & 1u) ^ 1u,
                                                                   abort_flag, a.status, a.limit));
                if (!ok) break;
                const uint32_t dst = sRing + slot * kDqSlot;
                const int live = u.Lk - t * 64;
                const bool zero = live < 64 && u.k0 + u.Lk < a.total_k;
                uint64_t *full = zero ? raw_full : &kv_full[slot];
                if (lane == 0) {
                    mbar_expect_tx(full, kDqSlot);
                    for (int h = 0; h < kHalves; ++h) {  // [K halves][V halves], 8 KB each
                        tma_load_3d(dst + h * 8192, &tk, full, 64 * h, u.hk, u.k0 + t * 64);
                        tma_load_3d(dst + kBlockBytes + h * 8192, &tv, full, 64 * h, u.hk, u.k0 + t * 64);
                    }
                }
                __syncwarp();
                if (zero) {  // the last tile of a sequence
                    ok = __all_sync(0xffffffffu, wait_plain(raw_full, tails++ & 1u, a.limit));
                    if (!ok) break;
                    zero_rows(sm + slot * kDqSlot, live, 64, 2 * kHalves, 8192, lane);
                    if (lane == 0) mbar_arrive(&kv_full[slot]);
                }
                ++seq;
            }
        }
        // drain: never leave with a copy in flight
        if (lane == 0)
            for (uint32_t s = seq > kDqRing ? seq - kDqRing : 0; s < seq; ++s)
                wait_plain(&kv_full[s % kDqRing], (s / kDqRing) & 1u, a.limit);
    } else if (warp == 1) {
        // ---------------- S / dP issuer (whole warp, one elected lane issues) ----------------
        constexpr uint32_t kIdS = idesc_bf16(128, 64, 0, 0);    // Q . K^T, dO . V^T
        auto off = [](int kk) { return static_cast<uint32_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4); };
        int slot = 0, b = 0;
        uint32_t kv_phase = 0, turn = 0, loaded = 0;  // turn: uses of the S buffers / 2; loaded: units with keys
        for (uint32_t n = 0; ok; ++n) {
            const int us = n & 1;
            ok = warp_wait(&u_full[us], (n >> 1) & 1u, abort_flag, a.status, a.limit);
            if (!ok) break;
            const int valid = units[us].valid, nt = units[us].nt;
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[us]);
            if (!valid) break;
            if (nt == 0) continue;
            ok = warp_wait(q_ready, loaded++ & 1u, abort_flag, a.status, a.limit);
            for (int t = 0; ok && t < nt; ++t) {
                ok = warp_wait(&kv_full[slot], kv_phase, abort_flag, a.status, a.limit);
                // both buffers are free once the dQ MMAs of their last tile have read its dS
                if (ok && turn > 0) ok = warp_wait(&s_free[b], (turn - 1) & 1u, abort_flag, a.status, a.limit);
                if (!ok) break;
                tc_fence_after();
                const uint32_t b0 = sRing + slot * kDqSlot;
                const uint32_t d = tmem + 64 * b;
                // descriptors advance by (byte offset >> 4) in their low address field
                const uint64_t dK = desc_sw128(b0, 16, 1024), dV = desc_sw128(b0 + kBlockBytes, 16, 1024);
                const uint32_t e = tmem + kDqColDP + 64 * b;
#pragma unroll
                for (int kk = 0; kk < D / 16; kk += 4)
                    mma_ts4_warp(d, d, d, d, tmem + kColQ + 8 * kk, tmem + kColQ + 8 * kk + 8,
                                 tmem + kColQ + 8 * kk + 16, tmem + kColQ + 8 * kk + 24, dK + off(kk),
                                 dK + off(kk + 1), dK + off(kk + 2), dK + off(kk + 3), kIdS, kk > 0, 1u);
#pragma unroll
                for (int kk = 0; kk < D / 16; kk += 4)
                    mma_ts4_warp(e, e, e, e, tmem + kColDO + 8 * kk, tmem + kColDO + 8 * kk + 8, tmem + kColDO + 8 * kk + 16,
                                 tmem + kColDO + 8 * kk + 24, dV + off(kk), dV + off(kk + 1), dV + off(kk + 2),
                                 dV + off(kk + 3), kIdS, kk > 0, 1u);
                mma_commit_warp(&s_full[b]);
                if (++slot == kDqRing) {
                    slot = 0;
                    kv_phase ^= 1u;
                }
                if (++b == 2) {
                    b = 0;
                    ++turn;
                }
            }
        }
        mma_commit_warp(sdp_done);  // completes once every MMA issued above has finished
        if (lane == 0) wait_plain(sdp_done, 0, a.limit);
        __syncwarp();
    } else if (warp == kDqGradWarp) {
        // ---------------- dQ issuer (whole warp, one elected lane issues) ----------------
        constexpr uint32_t kIdQ = idesc_bf16(128, D, 0, 1);     // dS . K (K MN-major)
        int slot = 0, b = 0;
        uint32_t phase = 0, ended = 0;
        for (uint32_t n = 0; ok; ++n) {
            const int us = n & 1;
            ok = warp_wait(&u_full[us], (n >> 1) & 1u, abort_flag, a.status, a.limit);
            if (!ok) break;
            const int valid = units[us].valid, nt = units[us].nt;
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[us]);
            if (!valid) break;
            if (nt == 0) continue;
            for (int t = 0; ok && t < nt; ++t) {
                ok = warp_wait(&ds_full[b], phase, abort_flag, a.status, a.limit);
                if (!ok) break;
                tc_fence_after();
                // K as the MN-major B operand: key k-step kk starts 2048 bytes further
                // and reads bf16 dS columns 32 (kk / 2) + 8 (kk % 2) of this tile's S
                const uint64_t gK = desc_sw128(sRing + slot * kDqSlot, 8192, 1024);
                const uint32_t c = tmem + 64 * b;
                mma_ts4_warp(tmem + kColDQ, tmem + kColDQ, tmem + kColDQ, tmem + kColDQ, c, c + 8, c + 32,
                             c + 40, gK, gK + 128, gK + 256, gK + 384, kIdQ, t > 0 ? 1u : 0u, 1u);
                mma_commit_warp(&kv_empty[slot]);
                mma_commit_warp(&s_free[b]);
                if (++slot == kDqRing) slot = 0;
                if (++b == 2) {
                    b = 0;
                    phase ^= 1u;
                }
            }
            if (ok) {
                mma_commit_warp(done);  // the unit's dQ is complete
                ++ended;
            }
        }
        if (!ok) {  // given up inside a unit: its MMAs still have to finish
            mma_commit_warp(done);
            ++ended;
        }
        if (lane == 0 && ended > 0) wait_plain(done, (ended - 1) & 1u, a.limit);
        __syncwarp();
    } else {
        // ---------------- dS warpgroups: row r, key half kg ----------------
        const int wq = warp & 3;                    // TMEM lane quarter of this warp
        const int kg = (warp - 2) >> 2;             // 0: keys 0-31, 1: keys 32-63
        const int r = wq * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        unsigned char *stage = sm + L::DQ_STAGE + (warp - 2) * 2048;
        const uint64_t c2 = f2_pack(a.c, a.c);
        uint32_t v32[D / 2];  // the next unit's Q row (group 0) or dO row (group 1)
        float nLr = 0.f, nDr = 0.f;
        // row of the unit in slot us: token and head, clamped to a real one
        auto place = [&](int us, int *tok, int *head) -> bool {
            const int rows = units[us].Lq * G, R0 = units[us].R0;
            const int row = min(R0 + r, rows - 1);
            *tok = row / G;
            *head = units[us].hk * G + row % G;
            return R0 + r < rows;
        };
        auto fetch = [&](int us) {
            int tok, head;
            place(us, &tok, &head);
            const int64_t prow = head * a.pad_rows + static_cast<int64_t>(units[us].pad) * 64 + tok;
            nLr = a.pad_l[prow];
            nDr = a.pad_d[prow];
            const uint4 *src = reinterpret_cast<const uint4 *>((kg ? a.dout : a.q).row(units[us].q0 + tok, head));
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
                const uint4 v = __ldg(src + e);
                v32[4 * e] = v.x;
                v32[4 * e + 1] = v.y;
                v32[4 * e + 2] = v.z;
                v32[4 * e + 3] = v.w;
            }
        };
        auto arrived = [&](uint32_t n) -> bool {  // the unit's description
            return __all_sync(0xffffffffu, wait_bar(&u_full[n & 1], (n >> 1) & 1u, abort_flag, a.status, a.limit));
        };
        int b = 0;
        uint32_t phase = 0, ended = 0, singles = 0;
        ok = ok && arrived(0);
        if (ok && units[0].valid && units[0].nt > 0) fetch(0);
        for (uint32_t n = 0; ok; ++n) {
            const int us = n & 1;
            if (!units[us].valid) break;
            const int nt = units[us].nt;
            const uint64_t nl2 = f2_pack(nLr, nLr), nd2 = f2_pack(nDr, nDr);
            int tok, head;
            const bool real = place(us, &tok, &head);
            const int64_t grow = units[us].q0 + tok;
            const int Lk = units[us].Lk, shift = Lk - units[us].Lq;
            int left = (a.causal ? min(Lk - 1, tok + shift) : Lk - 1) - 32 * kg;  // last key of this row
            int left0 = a.causal ? min(Lk - 1, units[us].R0 / G + shift) : Lk - 1;  // of the first row
            if (nt > 0) {
                // A operands of S and dP (the MMAs of the unit before have finished)
                const uint32_t col = kg ? kColDO : kColQ;
#pragma unroll
                for (int half = 0; half < D / 64; ++half)
                    tmem_st32(tmem + lane_base + col + 32 * half, reinterpret_cast<float *>(v32 + 32 * half));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
            }
            const bool few = left + 32 * kg < 64;  // all keys of this row are in the first tile
            // (two instances: a test for the first tile inside the loop cost it 8%)
            auto tile = [&](auto head) {
                ok = wait_bar(&s_full[b], phase, abort_flag, a.status, a.limit) && ok;
                tc_fence_after();
                const uint32_t scol = tmem + lane_base + b * 64 + 32 * kg;
                uint32_t gk[16];
                float sv[32], dp[32];
                tmem_ld32(scol, sv);
                tmem_ld32(scol + kDqColDP, dp);
                tmem_wait_ld();
                if (63 > left0) {  // masked tile: P = 0 and no NaN out of dP
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        sv[e] = e <= left ? sv[e] : -INFINITY;
                        dp[e] = e <= left ? dp[e] : 0.f;
                    }
                }
                if constexpr (head.value) {
                    // the first tile, where it holds all keys of some rows: their delta is the
                    // sum of P dP over it
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        sv[e] = fast_exp2(fmaf(sv[e], a.c, nLr));
                        sum = fmaf(sv[e], dp[e], sum);
                    }
                    float *red = reinterpret_cast<float *>(sm + L::DQ_RED);
                    red[128 * kg + r] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pair[wq]);
                    // (bounded, as every wait; the next write is behind the next unit's q_ready)
                    ok = wait_bar(&pair[wq], singles++ & 1u, abort_flag, a.status, a.limit) && ok;
                    sum = few ? sum + red[128 * (kg ^ 1) + r] : -nDr;
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        gk[e >> 1] = pack_bf16(sv[e] * (dp[e] - sum), sv[e + 1] * (dp[e + 1] - sum));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const uint64_t x = f2_fma(f2_pack(sv[e], sv[e + 1]), c2, nl2);
                        const uint64_t g = f2_mul(f2_pack(fast_exp2(f2_lo(x)), fast_exp2(f2_hi(x))),
                                                  f2_add(f2_pack(dp[e], dp[e + 1]), nd2));
                        gk[e >> 1] = pack_bf16(f2_lo(g), f2_hi(g));
                    }
                }
                // bf16 dS of keys [32 kg, 32 kg + 32) over this group's first 16 S columns
                tmem_st16(scol, gk);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_full[b]);
                if (++b == 2) {
                    b = 0;
                    phase ^= 1u;
                }
                left -= 64;
                left0 -= 64;
            };
            int t = 0;
            if (nt > 0 && left0 < 64) {
                tile(std::true_type{});
                t = 1;
            }
            for (; t < nt; ++t) tile(std::false_type{});
            // the next unit's rows travel while this one ends
            ok = __all_sync(0xffffffffu, ok);  // (lanes may have given up apart; the vote in `arrived` is the warp's)
            ok = ok && arrived(n + 1);
            ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
            if (!ok) break;
            if (units[us ^ 1].valid && units[us ^ 1].nt > 0) fetch(us ^ 1);
            // ---------------- epilogue: group kg writes dQ features [D/2 kg, +D/2) ----------------
            if (nt > 0) ok = wait_bar(done, ended++ & 1u, abort_flag, a.status, a.limit);
            tc_fence_after();
            ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
            if (!ok) break;
            __nv_bfloat16 *dst = real ? a.dq.row(grow, head) + (D / 2) * kg : nullptr;
#pragma unroll
            for (int part = 0; part < D / 64; ++part) {
                float v[32];
                if (nt > 0) {
                    tmem_ld32(tmem + lane_base + kColDQ + (D / 2) * kg + 32 * part, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                uint4 w[4];
#pragma unroll
                for (int e8 = 0; e8 < 4; ++e8) {
                    w[e8].x = pack_bf16(v[8 * e8] * a.scale, v[8 * e8 + 1] * a.scale);
                    w[e8].y = pack_bf16(v[8 * e8 + 2] * a.scale, v[8 * e8 + 3] * a.scale);
                    w[e8].z = pack_bf16(v[8 * e8 + 4] * a.scale, v[8 * e8 + 5] * a.scale);
                    w[e8].w = pack_bf16(v[8 * e8 + 6] * a.scale, v[8 * e8 + 7] * a.scale);
                }
                store_rows(stage, w, dst == nullptr ? nullptr : dst + 32 * part, lane);
            }
            tc_fence_before();  // dQ is read: the next unit's first dQ MMA may overwrite it
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[us]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    wait_for_prerequisites();  // the end of this launch is the end of the dK, dV one too
}

}  // namespace packed
}  // namespace nabla

template <int D>
static cudaError_t launch_packed_bwd(const nabla::packed::Args &a, int64_t q_tiles, int64_t key_tiles,
                                     cudaStream_t stream) {
    using namespace nabla::packed;
    cudaError_t err;
    {  // (without queries too: it looks at the borders)
        // heads a CTA of pre_kernel: 2 take 24 us at 100 MB, 1 27, 8 38; one where two
        // would not fill the GPU (six CTAs an SM)
        const int per = q_tiles * a.heads > 2 * 6 * kSms ? 2 : 1;
        pre_kernel<D><<<dim3(static_cast<unsigned>(q_tiles), (a.heads + per - 1) / per), kPreThreads, 0,
                        stream>>>(a, per);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    // without any query or key the maps only have to be valid: nothing is loaded
    const bool q = a.total_q > 0, k = a.total_k > 0;
    const View &any = q ? a.q : a.k;
    CUtensorMap mq, mdo, mk, mv, mv128;
    if (!nabla_make_tmap_view(&mq, q ? a.q : any, q ? a.total_q : 1, q ? a.heads : 1, D, 64, 1) ||
        !nabla_make_tmap_view(&mdo, q ? a.dout : any, q ? a.total_q : 1, q ? a.heads : 1, D, 64, 1) ||
        !nabla_make_tmap_view(&mk, k ? a.k : any, k ? a.total_k : 1, k ? a.heads_kv : 1, D, 64, 1) ||
        !nabla_make_tmap_view(&mv, k ? a.v : any, k ? a.total_k : 1, k ? a.heads_kv : 1, D, 64, 1) ||
        !nabla_make_tmap_view(&mv128, k ? a.v : any, k ? a.total_k : 1, k ? a.heads_kv : 1, D, 128, 1))
        return cudaErrorInvalidValue;
    if (k) {
        constexpr uint32_t kSmem = KvLayout<D>::kSmem;
        err = nabla_allow_smem<dkdv_kernel<D>>(kSmem);
        if (err != cudaSuccess) return err;
        err = nabla_launch_early(dkdv_kernel<D>, static_cast<unsigned>(key_tiles * a.heads_kv), kKvThreads, kSmem,
                                 stream, mq, mv128, mdo, a);
        if (err != cudaSuccess) return err;
    }
    if (q) {
        constexpr uint32_t kSmem = DqLayout<D>::kSmem;
        err = nabla_allow_smem<dq_kernel<D>>(kSmem);
        if (err != cudaSuccess) return err;
        const unsigned grid = static_cast<unsigned>(a.units < kSms ? a.units : kSms);
        if (k)
            return nabla_launch_early(dq_kernel<D>, grid, kDqThreads, kSmem, stream, mk, mv, a);
        dq_kernel<D><<<grid, kDqThreads, kSmem, stream>>>(mk, mv, a);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

// Upper bounds over the sequences: 64-row tiles of q, 128-key tiles (and, in
// a.units, 128-row tiles of the (token, head of a group) rows x heads_kv)
cudaError_t nabla_launch_packed_bwd(const nabla::packed::Args &a, int D, int64_t q_tiles,
                                    int64_t key_tiles, cudaStream_t stream) {
    return D == 128 ? launch_packed_bwd<128>(a, q_tiles, key_tiles, stream)
                    : launch_packed_bwd<64>(a, q_tiles, key_tiles, stream);
}
