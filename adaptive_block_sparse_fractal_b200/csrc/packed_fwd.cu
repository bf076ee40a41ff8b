// Attention of packed sequences, forward, on tcgen05 tensor cores (D = 128 or
// 64): o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys a row keeps.
//
// Work unit (one CTA): 256 rows of one sequence and one key head, as two
// tiles of 128.  Rows are (token, query head of the group) pairs, token major:
// row R is token R / G, head R % G of the G query heads that share the key
// head.  So every K/V tile serves all heads of the group, a short sequence
// still fills rows, and G need not divide anything.
//
// Per 128-key tile and row tile a:
//   S_a = Q_a . K^T    (both from shared memory, accumulator in TMEM)
//   P_a = exp2(S_a scale log2e - m)   one softmax warpgroup per row tile, one
//                      thread per row: no exchange between threads at all
//   O_a += P_a . V     (P_a in TMEM over S_a, V from shared memory)
// The tensor core alternates the row tiles (PV_0 S_0 PV_1 S_1 ...), so it works
// for one while the other is in its softmax.  P goes over in two halves of 64
// keys: the first half's MMAs run under the second half's exponentials.
//
// Rows keep a reference maximum; a row moves to a new one, and its O in TMEM
// is rescaled, only when a tile exceeds it by more than 2^8 (P is bf16 with a
// float32 accumulator, so the reference needs no more than that).  Statistics
// and sums are float32; P is rounded to bf16 (half a step, 2^-9 relative)
// because it is the tensor core's operand, the sum of a row is taken over the
// float32 values in front of that rounding.
//
// A tile that ends behind its sequence holds rows of the next one, or memory
// behind the last: their scores are replaced by -inf, and V's rows are zeroed
// in shared memory, as 0 * NaN would spread.
//
// Few rows against many keys (new tokens behind a cached context) leave the
// SMs idle: the key range is then split over gridDim.y and combine_kernel joins
// the parts.
//
// Warp roles (384 threads): warp 0 loads K and V by TMA, one thread of warp 1
// issues the MMAs, warps 4-7 and 8-11 are the softmax of row tiles 0 and 1
// (warps 2 and 3 only complete the first warpgroup).
// TMEM columns: S_0 [0,128), S_1 [128,256), O_0 [256, +D), O_1 [384, +D).
#include "packed.cuh"

namespace nabla {
namespace packed {

using namespace sm100;

constexpr int kFwdThreads = 384;
// Registers a thread: the launch gives 168 to each of the three warpgroups; the
// first (loads, MMA issue) hands some over to the softmax ones, whose rows of
// 128 scores need them: 80 + 2 * 208 = 496 <= 3 * 168.
constexpr int kRegsFew = 80, kRegsMany = 208;
constexpr int kTileKeys = 128;
constexpr int kRowsCta = 256;
constexpr float kFwdLn2 = 0.6931471805599453f;
constexpr float kHeadroom = 8.f;  // log2 a row may exceed its reference by

template <int D>
struct FwdLayout {
    static constexpr int kHalves = D / 64;
    static constexpr int kRing = D == 128 ? 5 : 9;
    static constexpr uint32_t kTile = 128u * D * 2;  // 128 rows x D bf16
    static constexpr uint32_t OFF_Q = 0;             // two row tiles
    static constexpr uint32_t OFF_RING = 2 * kTile;
    static constexpr uint32_t OFF_BAR = OFF_RING + kRing * kTile;
    static constexpr int kBars = 2 * kRing + 1 + 2 + 4 + 2 + 1 + 1;
    static constexpr uint32_t OFF_SEQ = OFF_BAR + 8 * kBars;
    static constexpr uint32_t OFF_SUM = (OFF_SEQ + sizeof(SeqTile) + 7) / 8 * 8;
    static constexpr uint32_t OFF_INT = OFF_SUM + 8 * (kFwdThreads / 32);
    static constexpr uint32_t kSmem = OFF_INT + 16 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ Args a) {
    using L = FwdLayout<D>;
    constexpr int kRing = L::kRing, kHalves = L::kHalves;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    unsigned char *sm = smem_raw + pad;
    const uint32_t sb = raw + pad;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
    uint64_t *kv_full = bar, *kv_empty = bar + kRing, *q_ready = bar + 2 * kRing;
    // per row tile: S complete; P halves written (four warps each); PV complete
    uint64_t *s_full = q_ready + 1, *p_full = s_full + 2, *pv_done = p_full + 4;
    uint64_t *raw_full = pv_done + 2;  // a tile that still has rows to zero
    uint64_t *all_done = raw_full + 1;
    SeqTile *st = reinterpret_cast<SeqTile *>(sm + L::OFF_SEQ);
    int *sInt = reinterpret_cast<int *>(sm + L::OFF_INT);  // [0] tmem base [2] abort
    volatile int *abort_flag = sInt + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group;

    const int64_t unit = blockIdx.x / a.heads_kv;
    const int hk = static_cast<int>(blockIdx.x % a.heads_kv);
    if (!find_seq<kFwdThreads>(
            a, unit, [=](int Lq, int) { return (Lq * G + kRowsCta - 1) / kRowsCta; },
            st, reinterpret_cast<int64_t *>(sm + L::OFF_SUM)))
        return;
    const int Lq = st->Lq, Lk = st->Lk, off = Lk - Lq;
    // the last tiles of a causal sequence keep the most keys: they go first
    const int rows = Lq * G;  // below 2^31: heads * total_q is
    const int R0 = ((rows + kRowsCta - 1) / kRowsCta - 1 - st->tile) * kRowsCta;

    // key tiles [j0, j0 + e[t]) of row tile t in this split
    int e[2], n[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = R0 + 128 * t;
        int kend = 0;
        if (first < rows) {
            const int last_tok = min(first + 127, rows - 1) / G;
            kend = a.causal ? min(Lk, last_tok + 1 + off) : Lk;
        }
        n[t] = kend > 0 ? (kend + kTileKeys - 1) / kTileKeys : 0;
    }
    const int nmax = max(n[0], n[1]);
    const int per = (nmax + gridDim.y - 1) / gridDim.y;
    const int j0 = min(nmax, static_cast<int>(blockIdx.y) * per), j1 = min(nmax, j0 + per);
#pragma unroll
    for (int t = 0; t < 2; ++t) e[t] = max(0, min(j1, n[t]) - j0);
    const int emax = max(e[0], e[1]);

    if (threadIdx.x == 0) {
        for (int r = 0; r < kRing; ++r) {
            mbar_init(&kv_full[r], 1);
            mbar_init(&kv_empty[r], 1);
        }
        mbar_init(q_ready, 8);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[2 * t], 4);
            mbar_init(&p_full[2 * t + 1], 4);
            mbar_init(&pv_done[t], 1);
        }
        mbar_init(raw_full, 1);
        mbar_init(all_done, 1);
        sInt[2] = *reinterpret_cast<volatile int *>(a.status) != 0 ? 1 : 0;
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

    if (warp < 4) {
    reg_dealloc<kRegsFew>();
    if (warp == 0) {
        // ---------------- K and V tiles in the order the MMAs take them ----------------
        if (lane == 0) {
            prefetch_tmap(&tk);
            prefetch_tmap(&tv);
        }
        uint32_t seq = 0;
        auto load = [&](const CUtensorMap *tm, int j, bool is_v) -> bool {
            const int slot = static_cast<int>(seq % kRing);
            // V's rows behind the sequence (the map zero-fills those behind the tensor)
            const int live = Lk - j * kTileKeys;
            const bool zero = is_v && live < kTileKeys && st->k0 + Lk < a.total_k;
            const bool ok = __all_sync(
                0xffffffffu, lane != 0 || wait_bar(&kv_empty[slot], ((seq / kRing) & 1u) ^ 1u,
                                                   abort_flag, a.status, a.limit));
            if (!ok) return false;
            const uint32_t dst = sb + L::OFF_RING + slot * kTile;
            uint64_t *full = zero ? raw_full : &kv_full[slot];
            if (lane == 0) {
                mbar_expect_tx(full, kTile);
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    tma_load_3d(dst + h * 16384, tm, full, 64 * h, hk, st->k0 + j * kTileKeys);
            }
            __syncwarp();
            if (zero) {  // at most once: the last tile
                const bool in = wait_plain(raw_full, 0, a.limit);
                if (!__all_sync(0xffffffffu, in)) return false;
                zero_rows(sm + L::OFF_RING + slot * kTile, live, kTileKeys, kHalves, 16384, lane);
                if (lane == 0) mbar_arrive(&kv_full[slot]);
            }
            ++seq;
            return true;
        };
        if (emax > 0 && !*abort_flag) {
            bool ok = load(&tk, j0, false);
            for (int i = 1; ok && i < emax; ++i)
                ok = load(&tv, j0 + i - 1, true) && load(&tk, j0 + i, false);
            if (ok) load(&tv, j0 + emax - 1, true);
        }
        // drain: never leave with a copy in flight
        if (lane == 0)
            for (uint32_t s = seq > kRing ? seq - kRing : 0; s < seq; ++s)
                wait_plain(&kv_full[s % kRing], (s / kRing) & 1u, a.limit);
    } else if (warp == 1) {
        // ---------------- MMA issuer (one thread) ----------------
        if (lane == 0) {
            constexpr uint32_t kIdS = idesc_bf16(128, 128, 0, 0);
            constexpr uint32_t kIdPV = idesc_bf16(128, D, 0, 1);
            uint32_t have = 0;  // ring entries known to have arrived: [0, have)
            auto arrived = [&](uint32_t s) -> bool {
                if (s < have) return true;
                if (!wait_bar(&kv_full[s % kRing], (s / kRing) & 1u, abort_flag, a.status, a.limit))
                    return false;
                have = s + 1;
                return true;
            };
            // tile i: K is ring entry 0 for i = 0 and 2i after (K0 V0 K1 V1 ...): entry 2i; V: 2i + 1
            auto S = [&](int t, int i) -> bool {
                const uint32_t s = 2u * i;
                if (!arrived(s)) return false;
                tc_fence_after();
                const uint32_t kb = sb + L::OFF_RING + (s % kRing) * kTile;
                const uint32_t qb = sb + L::OFF_Q + t * kTile;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
                    mma_ss_1(tmem + 128 * t, desc_sw128(qb + o, 16, 1024),
                             desc_sw128(kb + o, 16, 1024), kIdS, kk > 0);
                }
                mma_commit_1(&s_full[t]);
                return true;
            };
            auto PV = [&](int t, int i) -> bool {
                const uint32_t s = 2u * i + 1;
                if (!arrived(s)) return false;
                const uint32_t vb = sb + L::OFF_RING + (s % kRing) * kTile;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait_bar(&p_full[2 * t + half], i & 1, abort_flag, a.status, a.limit))
                        return false;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                        mma_ts_1(tmem + 256 + 128 * t, tmem + 128 * t + 8 * kk,
                                 desc_sw128(vb + kk * 2048, 16384, 1024), kIdPV, (i > 0 || kk > 0));
                }
                mma_commit_1(&pv_done[t]);
                return true;
            };
            if (emax > 0 && !*abort_flag &&
                wait_bar(q_ready, 0, abort_flag, a.status, a.limit)) {
                bool ok = true;
                for (int t = 0; ok && t < 2; ++t)
                    if (e[t] > 0) ok = S(t, 0);
                if (ok) mma_commit_1(&kv_empty[0]);
                for (int i = 0; ok && i < emax; ++i) {
                    for (int t = 0; ok && t < 2; ++t) {
                        if (i >= e[t]) continue;
                        ok = PV(t, i);
                        if (ok && (t == 1 || i >= e[1])) mma_commit_1(&kv_empty[(2 * i + 1) % kRing]);
                        if (ok && i + 1 < e[t]) ok = S(t, i + 1);
                    }
                    if (ok && i + 1 < emax) mma_commit_1(&kv_empty[(2 * i + 2) % kRing]);
                }
            }
            // completes once every MMA issued above has finished
            mma_commit_1(all_done);
            wait_plain(all_done, 0, a.limit);
        }
    }
    } else {
        reg_alloc<kRegsMany>();
        // ---------------- softmax: thread = row ----------------
        const int t = (warp - 4) >> 2;
        const int wq = warp & 3;
        const int r = wq * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        const bool real = R0 + 128 * t + r < rows;
        const int row = min(R0 + 128 * t + r, rows - 1);
        const int tok = row / G;
        const int head = hk * G + row % G;
        {
            // Q rows of this warp -> shared memory; D/8 threads take one row's 16-byte chunks
            constexpr int kChunks = D / 8, kRowsStep = 32 / kChunks;
            const int c = lane % kChunks;
            unsigned char *qt = sm + L::OFF_Q + t * kTile + (c >> 3) * 16384;
#pragma unroll 4
            for (int rr = lane / kChunks; rr < 32; rr += kRowsStep) {
                const int lr = wq * 32 + rr;
                const int gr = R0 + 128 * t + lr;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (gr < rows)
                    v = __ldg(reinterpret_cast<const uint4 *>(
                            a.q.row(st->q0 + gr / G, hk * G + gr % G)) + c);
                *reinterpret_cast<uint4 *>(qt + lr * 128 + (((c & 7) ^ (lr & 7)) << 4)) = v;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);
        }
        const int lim = a.causal ? min(Lk - 1, tok + off) : Lk - 1;  // last key of this row
        // the first row of the tile keeps the fewest: key tiles from here on are masked
        const int lim0 = a.causal ? min(Lk - 1, (R0 + 128 * t) / G + off) : Lk - 1;
        const uint32_t scol = tmem + lane_base + 128 * t, ocol = tmem + lane_base + 256 + 128 * t;
        const float c = a.c;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        const int et = *abort_flag ? 0 : (t ? e[1] : e[0]);
        for (int i = 0; i < et; ++i) {
            ok = wait_bar(&s_full[t], i & 1, abort_flag, a.status, a.limit) && ok;
            tc_fence_after();
            float s[128];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld32(scol + 32 * q, s + 32 * q);
            tmem_wait_ld();
            const int kb = (j0 + i) * kTileKeys;
            if (kb + kTileKeys - 1 > lim0) {
                const int left = lim - kb;
#pragma unroll
                for (int k = 0; k < 128; ++k) s[k] = k <= left ? s[k] : -INFINITY;
            }
            float mx[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) mx[q] = s[q];
#pragma unroll
            for (int k = 8; k < 128; k += 2) mx[(k >> 1) & 7] = fmax3(mx[(k >> 1) & 7], s[k], s[k + 1]);
            const float tmax = c * fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                         fmaxf(mx[6], mx[7]));
            // warp-uniform decision: the TMEM accesses below are collective
            if (__any_sync(0xffffffffu, tmax > m + kHeadroom)) {
                const float mnew = fmaxf(m, tmax);
                const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - mnew);
                if (i > 0) {
                    ok = wait_bar(&pv_done[t], (i - 1) & 1, abort_flag, a.status, a.limit) && ok;
                    tc_fence_after();
#pragma unroll
                    for (int part = 0; part < D / 32; ++part) {
                        float ov[32];
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; ++q) ov[q] *= alpha;
                        tmem_st32(ocol + 32 * part, ov);
                    }
                    tmem_wait_st();
                }
                l *= alpha;
                m = mnew;
            }
            const float mref = m == -INFINITY ? 0.f : m;  // rows without a key so far
            const uint64_t c2 = f2_pack(c, c), nm2 = f2_pack(-mref, -mref);
            uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    const uint64_t x = f2_fma(f2_pack(s[64 * half + k], s[64 * half + k + 1]), c2, nm2);
                    const float p0 = fast_exp2(f2_lo(x)), p1 = fast_exp2(f2_hi(x));
                    ls2[(k >> 1) & 3] = f2_add(ls2[(k >> 1) & 3], f2_pack(p0, p1));
                    pk[k >> 1] = pack_bf16(p0, p1);
                }
                tmem_st32(scol + 32 * half, reinterpret_cast<float *>(pk));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
            }
            const uint64_t ls = f2_add(f2_add(ls2[0], ls2[1]), f2_add(ls2[2], ls2[3]));
            l += f2_lo(ls) + f2_hi(ls);
        }
        // ---------------- epilogue ----------------
        if (ok && et > 0) ok = wait_bar(&pv_done[t], (et - 1) & 1, abort_flag, a.status, a.limit);
        tc_fence_after();
        const bool aborted = __any_sync(0xffffffffu, *abort_flag != 0);
        const bool read_o = !aborted && et > 0 && __all_sync(0xffffffffu, ok);
        if (!aborted) {
            const int64_t grow = st->q0 + tok;
            const bool live = l > 0.f;
            if (gridDim.y == 1) {
                if (real && a.lse != nullptr)
                    a.lse[head * a.total_q + grow] = live ? (m + log2f(l)) * kFwdLn2 : l == 0.f ? -INFINITY : l;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                __nv_bfloat16 *dst = a.o.row(grow, head);
#pragma unroll
                for (int part = 0; part < D / 32; ++part) {
                    float ov[32];
                    if (read_o) {
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
                    }
                    if (!read_o || l == 0.f) {
#pragma unroll
                        for (int q = 0; q < 32; ++q) ov[q] = 0.f;
                    }
                    if (real) {
#pragma unroll
                        for (int e8 = 0; e8 < 4; ++e8) {
                            uint4 w;
                            w.x = pack_bf16(ov[8 * e8] * inv, ov[8 * e8 + 1] * inv);
                            w.y = pack_bf16(ov[8 * e8 + 2] * inv, ov[8 * e8 + 3] * inv);
                            w.z = pack_bf16(ov[8 * e8 + 4] * inv, ov[8 * e8 + 5] * inv);
                            w.w = pack_bf16(ov[8 * e8 + 6] * inv, ov[8 * e8 + 7] * inv);
                            *reinterpret_cast<uint4 *>(dst + 32 * part + 8 * e8) = w;
                        }
                    }
                }
            } else {
                // unnormalised part of this split: [split][token][head][D], then (m, l)
                const int64_t slot = (static_cast<int64_t>(blockIdx.y) * a.total_q + grow) * a.heads + head;
                float *dst = a.part + slot * D;
                if (real)
                    reinterpret_cast<float2 *>(a.part + static_cast<int64_t>(gridDim.y) * a.total_q * a.heads * D)[slot] =
                        make_float2(m, l);
#pragma unroll
                for (int part = 0; part < D / 32; ++part) {
                    float ov[32];
                    if (read_o) {
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q) ov[q] = 0.f;
                    }
                    if (real) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<float4 *>(dst + 32 * part + q) =
                                make_float4(ov[q], ov[q + 1], ov[q + 2], ov[q + 3]);
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

// Joins the parts of the splits: one warp per (token, head) row.  Rows that
// belong to no sequence are left alone.
template <int D>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ Args a, int splits) {
    if (*reinterpret_cast<volatile int *>(a.status) != 0) return;
    const int lane = threadIdx.x & 31;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (id >= a.total_q * a.heads) return;
    const int64_t tok = id / a.heads;
    const int head = static_cast<int>(id % a.heads);
    // does any sequence hold this token?  (borders ascend)
    if (tok < a.cu_q[0] || tok >= a.cu_q[a.seqs]) return;
    const int64_t slots = a.total_q * a.heads;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part + splits * slots * D);
    float m = -INFINITY;
    for (int s = 0; s < splits; ++s) m = fmaxf(m, ml[s * slots + id].x);
    const float mref = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
    for (int s = 0; s < splits; ++s) {
        const float2 v = ml[s * slots + id];
        const float w = exp2f(v.x - mref);
        l += v.y * w;
        const float *p = a.part + (s * slots + id) * D + lane * (D / 32);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] += p[e] * w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat16 *dst = a.o.row(tok, head) + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2)
        *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && a.lse != nullptr)
        a.lse[head * a.total_q + tok] = l > 0.f ? (mref + log2f(l)) * kFwdLn2 : l == 0.f ? -INFINITY : l;
}

}  // namespace packed
}  // namespace nabla

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
typedef CUresult (*NablaEncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                       const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                       const cuuint32_t *, CUtensorMapInterleave,
                                       CUtensorMapSwizzle, CUtensorMapL2promotion,
                                       CUtensorMapFloatOOBfill);

bool nabla_make_tmap_view(CUtensorMap *m, const nabla::packed::View &v, int64_t tokens, int heads,
                          int D, int rows) {
    static const NablaEncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<NablaEncodeTiledFn>(p);
    }();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    // a dimension of size one has no distance of its own
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? v.head : D) * 2,
                                   static_cast<cuuint64_t>(tokens > 1 ? v.token : D) * 2};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.p, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static cudaError_t launch_packed_fwd(const nabla::packed::Args &a, int64_t units, int splits,
                                     cudaStream_t stream) {
    using namespace nabla::packed;
    CUtensorMap mk, mv;
    // without any key nothing is loaded; the map only has to be valid
    const bool keys = a.total_k > 0;
    if (!nabla_make_tmap_view(&mk, keys ? a.k : a.q, keys ? a.total_k : 1, keys ? a.heads_kv : 1, D, 128) ||
        !nabla_make_tmap_view(&mv, keys ? a.v : a.q, keys ? a.total_k : 1, keys ? a.heads_kv : 1, D, 128))
        return cudaErrorInvalidValue;
    constexpr uint32_t kSmem = FwdLayout<D>::kSmem;
    cudaError_t err = cudaFuncSetAttribute(fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    fwd_kernel<D><<<dim3(static_cast<unsigned>(units), splits), kFwdThreads, kSmem, stream>>>(mk, mv, a);
    err = cudaGetLastError();
    if (err != cudaSuccess || splits == 1) return err;
    const int64_t rows = a.total_q * a.heads;
    combine_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a, splits);
    return cudaGetLastError();
}

// units: (256-row tiles, an upper bound over the sequences) x heads_kv
cudaError_t nabla_launch_packed_fwd(const nabla::packed::Args &a, int D, int64_t units, int splits,
                                    cudaStream_t stream) {
    return D == 128 ? launch_packed_fwd<128>(a, units, splits, stream)
                    : launch_packed_fwd<64>(a, units, splits, stream);
}
