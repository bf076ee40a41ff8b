// Attention of packed sequences, forward, on tcgen05 tensor cores (D = 128 or
// 64): o_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys a row keeps.
//
// Work unit: two row tiles of one sequence and one key head.  The rows of a tile
// are (token, query head of the group) pairs, token major: floor(128 / G)
// tokens of the G query heads that share the key head, which is one TMA box of
// [tokens][G][64 features] and leaves at most G - 1 of the 128 rows of the MMA
// idle.  So every K/V tile serves all heads of the group and a short sequence
// still fills rows.
//
// Per 128-key tile and row tile t:
//   S_t = Q_t . K^T    (both from shared memory, accumulator in TMEM)
//   P_t = exp2(S_t scale log2e - m)   one softmax warpgroup per row tile, one
//                      thread per row: no exchange between threads at all
//   O_t += P_t . V     (P_t in TMEM over S_t, V from shared memory)
// The tensor core works for one row tile while the other is in its softmax.
//
// At D = 128 a tile costs the tensor core 1,024 cycles and its 16,384
// exponentials the SFU another 1,024 (16 a cycle and SM), so part of them is
// taken on the FMA pipe instead: 2^x = 2^n p(x - n), n the nearest integer, p
// the degree-4 polynomial that minimises the largest relative error of 2^f on
// [-1/2, 1/2] (2.6e-6, found with a Remez iteration; P is rounded to bf16, at
// 2e-3, next).
//
// A row's reference is the maximum of its first tile.  Later tiles are taken
// against it without looking for their own maximum: P (bf16) and the float32
// sums have the exponent range for it.  Only when a tile's sum passes 2^16 is it
// taken again, against its true maximum, to which O (in TMEM) and the sum
// then move.  That leaves the loop with five instructions a pair of scores.
// Statistics and sums are float32; P is rounded to bf16 (half a step, 2^-8
// relative) because it is the tensor core's operand, the sum of a row is taken
// over the float32 values in front of that rounding.
//
// A tile that ends behind its sequence holds rows of the next one, or memory
// behind the last: their scores are replaced by -inf, and V's rows are zeroed
// in shared memory, as 0 * NaN would spread.  (A NaN or infinity in a row of V
// that a causal row does not keep, but another row of its sequence does, may
// still reach the rows whose tile touches it.)
//
// The kernel is persistent: one CTA an SM takes units from a counter until none
// is left, loading the next unit's Q, K and V while the softmax warps finish
// the last one.  Which CTA takes a unit does not change its result.
//
// Few rows against many keys (new tokens behind a cached context) leave the
// SMs idle: the key range is then split and combine_kernel joins the parts.
//
// Warp roles (384 threads): warp 0 takes units and loads by TMA, warps 1 and 2
// issue the MMAs of row tiles 0 and 1, warps 4-7 and 8-11 are their softmax
// (warp 3 only completes the first warpgroup).  The issuing warps stay converged
// and send four MMAs per elect.sync (a lone lane takes about as long to issue an
// MMA as it runs).  They take turns, PV_0 S_0 then PV_1 S_1, each waiting for its
// operands before its turn: the MMAs of a turn go out in one run, and the row
// tiles stay half a period apart (free-running issuers fell into step, both
// in their softmax and then both at the tensor core, and lost 15%).
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
constexpr float kFwdLn2 = 0.6931471805599453f;
constexpr float kMaxSum = 65536.f;  // largest sum of a row's P over a tile against an old reference
constexpr int kPolyOf8 = 3;       // pairs of every 8 whose exponentials the FMA pipe takes

// One unit, as the loading warp hands it to the others.
struct Unit {
    int valid, hk, split;
    int q0, Lq, k0, Lk;
    int tok0;     // first token of row tile 0
    int j0;       // first key tile of this split
    int e[2];     // key tiles of each row tile in it
};

template <int D>
struct FwdLayout {
    static constexpr int kHalves = D / 64;
    static constexpr int kRing = D == 128 ? 5 : 9;
    static constexpr uint32_t kTile = 128u * D * 2;  // 128 rows x D bf16
    static constexpr uint32_t OFF_Q = 0;             // two row tiles
    static constexpr uint32_t OFF_RING = 2 * kTile;
    static constexpr uint32_t OFF_BAR = OFF_RING + kRing * kTile;
    static constexpr int kBars = 2 * kRing + 4 + 2 + 2 + 2 + 4 + 1 + 4;
    static constexpr uint32_t OFF_UNIT = OFF_BAR + 8 * kBars;
    static constexpr uint32_t OFF_INT = OFF_UNIT + 2 * sizeof(Unit);
    static constexpr uint32_t kSmem = OFF_INT + 16 + 1024;
};

// 2^x for both halves of a pair, x finite and <= about 2^8, on the FMA pipe
__device__ __forceinline__ void exp2_poly(uint64_t x, float &p0, float &p1) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    const uint64_t big = f2_pack(kRound, kRound), nbig = f2_pack(-kRound, -kRound);
    x = f2_pack(fmaxf(f2_lo(x), -126.f), fmaxf(f2_hi(x), -126.f));
    const uint64_t t = f2_add(x, big);
    const uint64_t f = f2_fma(f2_add(t, nbig), f2_pack(-1.f, -1.f), x);
    uint64_t p = f2_fma(f2_pack(0.009570101911165427f, 0.009570101911165427f), f,
                        f2_pack(0.055917860319388245f, 0.055917860319388245f));
    p = f2_fma(p, f, f2_pack(0.2402474482786378f, 0.2402474482786378f));
    p = f2_fma(p, f, f2_pack(0.6931218147366892f, 0.6931218147366892f));
    p = f2_fma(p, f, f2_pack(0.9999992614457122f, 0.9999992614457122f));
    // the integer stands in the low bits of t: into the exponent
    p0 = __uint_as_float(static_cast<uint32_t>(p) + (static_cast<uint32_t>(t) << 23));
    p1 = __uint_as_float(static_cast<uint32_t>(p >> 32) + (static_cast<uint32_t>(t >> 32) << 23));
}

// P of 32 keys from their scores, as packed bf16; adds the values to four sums.
template <int kPoly>
__device__ __forceinline__ void softmax_part(const float *s, uint64_t c2, uint64_t nm2,
                                             uint64_t *ls2, uint32_t *pk) {
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        const uint64_t x = f2_fma(f2_pack(s[k], s[k + 1]), c2, nm2);
        float p0, p1;
        // spread over the row, so that both pipes are busy at once
        if (((k >> 1) * kPoly) % 8 + kPoly > 7 && kPoly > 0) {
            exp2_poly(x, p0, p1);
        } else {
            p0 = fast_exp2(f2_lo(x));
            p1 = fast_exp2(f2_hi(x));
        }
        ls2[(k >> 1) & 3] = f2_add(ls2[(k >> 1) & 3], f2_pack(p0, p1));
        pk[k >> 1] = pack_bf16(p0, p1);
    }
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, const __grid_constant__ Args a) {
    using L = FwdLayout<D>;
    constexpr int kRing = L::kRing, kHalves = L::kHalves;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    unsigned char *sm = smem_raw + pad;
    const uint32_t sb = raw + pad;
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
    uint64_t *kv_full = bar, *kv_empty = bar + kRing;
    uint64_t *q_full = bar + 2 * kRing, *q_empty = q_full + 2;  // per row tile
    // per row tile: S complete; P written (its four warps); PV complete
    uint64_t *s_full = q_empty + 2, *p_full = s_full + 2, *pv_done = p_full + 2;
    // per unit slot: written by the loading warp; read by the ten others
    uint64_t *u_full = pv_done + 2, *u_empty = u_full + 2;
    uint64_t *raw_full = u_empty + 2;  // a tile that still has rows to zero
    uint64_t *all_done = raw_full + 1, *turn = all_done + 2;  // per issuing warp
    volatile Unit *units = reinterpret_cast<Unit *>(sm + L::OFF_UNIT);
    int *sInt = reinterpret_cast<int *>(sm + L::OFF_INT);  // [0] tmem base [2] abort
    volatile int *abort_flag = sInt + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group, tpt = a.tile_tokens;  // tokens a row tile

    if (threadIdx.x == 0) {
        for (int r = 0; r < kRing; ++r) {
            mbar_init(&kv_full[r], 1);
            mbar_init(&kv_empty[r], 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_empty[t], 1);
            mbar_init(&all_done[t], 1);
            mbar_init(&turn[t], 1);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&pv_done[t], 1);
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 10);
        }
        mbar_init(raw_full, 1);
        sInt[2] = *reinterpret_cast<volatile int *>(a.status) != 0 ? 1 : 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(&sInt[0]), 512);
        tmem_relinquish();
    }
    // every CTA looks at every border before anything is written
    const bool good = borders_ok(a);
    tc_fence_before();
    const bool go = !__syncthreads_or(!good);
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(sInt[0]);
    if (!go) {
        if (threadIdx.x == 0) atomicExch(a.status, kDevParam);
    } else if (warp < 4) {
        reg_dealloc<kRegsFew>();
        if (warp == 0) {
            // ---------------- units, then their Q, K and V in the order the MMAs take them ----------------
            if (lane == 0) {
                prefetch_tmap(&tq);
                prefetch_tmap(&tk);
                prefetch_tmap(&tv);
            }
            uint32_t seq = 0, tails = 0, nq[2] = {0, 0};
            bool ok = __all_sync(0xffffffffu, *abort_flag == 0);
            auto load = [&](const Unit &u, const CUtensorMap *tm, int j, bool is_v) {
                const int slot = static_cast<int>(seq % kRing);
                // V's rows behind the sequence (the map zero-fills those behind the tensor)
                const int live = u.Lk - j * kTileKeys;
                const bool zero = is_v && live < kTileKeys && u.k0 + u.Lk < a.total_k;
                ok = ok && __all_sync(0xffffffffu,
                                      lane != 0 || wait_bar(&kv_empty[slot], ((seq / kRing) & 1u) ^ 1u,
                                                            abort_flag, a.status, a.limit));
                if (!ok) return;
                const uint32_t dst = sb + L::OFF_RING + slot * kTile;
                uint64_t *full = zero ? raw_full : &kv_full[slot];
                if (lane == 0) {
                    mbar_expect_tx(full, kTile);
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        tma_load_3d(dst + h * 16384, tm, full, 64 * h, u.hk, u.k0 + j * kTileKeys);
                }
                __syncwarp();
                if (zero) {  // the last tile of a sequence
                    ok = __all_sync(0xffffffffu, wait_plain(raw_full, tails++ & 1u, a.limit));
                    if (!ok) return;
                    zero_rows(sm + L::OFF_RING + slot * kTile, live, kTileKeys, kHalves, 16384, lane);
                    if (lane == 0) mbar_arrive(&kv_full[slot]);
                }
                ++seq;
            };
            UnitScan scan;
            int64_t x = lane == 0 ? take_unit(a) : 0;
            for (uint32_t n = 0; ok; ++n) {
                x = __shfl_sync(0xffffffffu, x, 0);
                const int64_t now = x;
                if (lane == 0) x = take_unit(a);  // the next one, under this one's loads
                Unit u = {};
                const int64_t ux = now / a.splits;
                int tile;
                u.split = static_cast<int>(now % a.splits);
                u.hk = static_cast<int>(ux % a.heads_kv);
                u.valid = scan.find(a, ux / a.heads_kv, 2 * tpt, lane, &u.q0, &u.Lq, &u.k0, &u.Lk, &tile);
                int emax = 0;
                if (u.valid) {
                    // the last tiles of a causal sequence keep the most keys: they go first
                    u.tok0 = ((u.Lq + 2 * tpt - 1) / (2 * tpt) - 1 - tile) * 2 * tpt;
                    const int off = u.Lk - u.Lq;
                    int kt[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int first = u.tok0 + t * tpt;
                        const int last = min(first + tpt, u.Lq) - 1;
                        const int kend = first >= u.Lq ? 0 : a.causal ? min(u.Lk, last + 1 + off) : u.Lk;
                        kt[t] = kend > 0 ? (kend + kTileKeys - 1) / kTileKeys : 0;
                    }
                    const int all = max(kt[0], kt[1]), per = (all + a.splits - 1) / a.splits;
                    u.j0 = min(all, u.split * per);
                    const int j1 = min(all, u.j0 + per);
                    u.e[0] = max(0, min(j1, kt[0]) - u.j0);
                    u.e[1] = max(0, min(j1, kt[1]) - u.j0);
                    emax = max(u.e[0], u.e[1]);
                }
                const int us = n & 1;
                ok = __all_sync(0xffffffffu, lane != 0 || wait_bar(&u_empty[us], ((n >> 1) & 1u) ^ 1u, abort_flag,
                                                                   a.status, a.limit));
                if (!ok) break;
                if (lane == 0) {
                    volatile Unit &w = units[us];
                    w.valid = u.valid;
                    w.hk = u.hk;
                    w.split = u.split;
                    w.q0 = u.q0;
                    w.Lq = u.Lq;
                    w.k0 = u.k0;
                    w.Lk = u.Lk;
                    w.tok0 = u.tok0;
                    w.j0 = u.j0;
                    w.e[0] = u.e[0];
                    w.e[1] = u.e[1];
                    mbar_arrive(&u_full[us]);
                }
                __syncwarp();
                if (!u.valid) break;
                if (emax == 0) continue;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (u.e[t] == 0 || !ok) continue;
                    ok = __all_sync(0xffffffffu, lane != 0 || wait_bar(&q_empty[t], (nq[t] & 1u) ^ 1u, abort_flag,
                                                                       a.status, a.limit));
                    if (!ok) continue;
                    ++nq[t];
                    if (lane == 0) {
                        mbar_expect_tx(&q_full[t], static_cast<uint32_t>(tpt * G) * 128u * kHalves);
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            tma_load_3d(sb + L::OFF_Q + t * kTile + h * 16384, &tq, &q_full[t], 64 * h, u.hk * G,
                                        u.q0 + u.tok0 + t * tpt);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                load(u, &tk, u.j0, false);
                for (int i = 1; ok && i < emax; ++i) {
                    load(u, &tv, u.j0 + i - 1, true);
                    if (ok) load(u, &tk, u.j0 + i, false);
                }
                if (ok) load(u, &tv, u.j0 + emax - 1, true);
            }
            // drain: never leave with a copy in flight
            if (lane == 0) {
                for (int t = 0; t < 2; ++t)
                    if (nq[t] > 0) wait_plain(&q_full[t], (nq[t] - 1) & 1u, a.limit);
                for (uint32_t s = seq > kRing ? seq - kRing : 0; s < seq; ++s)
                    wait_plain(&kv_full[s % kRing], (s / kRing) & 1u, a.limit);
            }
        } else if (warp < 3) {
            // ---------------- MMA issuer of row tile t (the whole warp, converged) ----------------
            const int t = warp - 1;
            constexpr uint32_t kIdS = idesc_bf16(128, 128, 0, 0);
            constexpr uint32_t kIdPV = idesc_bf16(128, D, 0, 1);
            const uint32_t ds = tmem + 128 * t, dov = tmem + 256 + 128 * t;
            const uint64_t qd = desc_sw128(sb + L::OFF_Q + t * kTile, 16, 1024);
            uint32_t slot = 0, phase = 0;  // next ring entry: K0 V0 K1 V1 ... of one unit after another
            uint32_t np = 0, nq = 0;       // tiles and units this row tile has seen
            uint32_t turns = t ^ 1u;       // parity of the next turn; row tile 0 has the first
            bool ok = __all_sync(0xffffffffu, *abort_flag == 0);
            auto next = [&]() {
                if (++slot == kRing) {
                    slot = 0;
                    phase ^= 1u;
                }
            };
            auto arrived = [&]() -> bool {
                return warp_wait(&kv_full[slot], phase, abort_flag, a.status, a.limit);
            };
            auto my_turn = [&]() -> bool {
                const bool got = warp_wait(&turn[t], turns, abort_flag, a.status, a.limit);
                turns ^= 1u;
                return got;
            };
            auto pass_turn = [&]() {
                if (lane == 0) mbar_arrive(&turn[t ^ 1]);
                __syncwarp();
            };
            auto S = [&]() {
                const uint64_t kd = desc_sw128(sb + L::OFF_RING + slot * kTile, 16, 1024);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const uint32_t o = h * 1024;  // halves 16 KB, 16 features 32 bytes
                    mma_ss4_warp(ds, ds, ds, ds, qd + o, qd + o + 2, qd + o + 4, qd + o + 6, kd + o, kd + o + 2,
                                 kd + o + 4, kd + o + 6, kIdS, h > 0, 1u);
                }
            };
            for (uint32_t n = 0; ok; ++n) {
                const int us = n & 1;
                ok = warp_wait(&u_full[us], (n >> 1) & 1u, abort_flag, a.status, a.limit);
                if (!ok) break;
                const int valid = units[us].valid;
                const int e = units[us].e[t], emax = max(e, units[us].e[t ^ 1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&u_empty[us]);
                if (!valid) break;
                if (emax == 0) continue;
                // turn -1: S(0); turn i: PV(i), S(i + 1).  All waits of a turn
                // stand in front of it, so that its MMAs go out in one run.
                if (e > 0) {
                    ok = warp_wait(&q_full[t], nq & 1u, abort_flag, a.status, a.limit);
                    ++nq;
                }
                ok = ok && arrived() && my_turn();
                if (!ok) break;
                tc_fence_after();
                if (e > 0) {
                    S();
                    mma_commit_warp(&s_full[t]);
                    mma_commit_warp(&kv_empty[slot]);
                    if (e == 1) mma_commit_warp(&q_empty[t]);
                } else if (lane == 0) {
                    mbar_arrive(&kv_empty[slot]);
                }
                pass_turn();
                next();
                for (int i = 0; ok && i < emax; ++i) {
                    const bool more = i + 1 < emax;
                    ok = arrived();  // V(i)
                    const uint32_t vslot = slot;
                    next();
                    if (ok && more) ok = arrived();  // K(i + 1)
                    if (ok && i < e) {
                        ok = warp_wait(&p_full[t], np & 1u, abort_flag, a.status, a.limit);
                        ++np;
                    }
                    ok = ok && my_turn();
                    if (!ok) break;
                    tc_fence_after();
                    if (i < e) {
                        const uint64_t vd = desc_sw128(sb + L::OFF_RING + vslot * kTile, 16384, 1024);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            // 16 keys: 8 columns of P, 2 KB of V
                            const uint32_t p = ds + 32 * half;
                            const uint64_t b = vd + 512 * half;
                            mma_ts4_warp(dov, dov, dov, dov, p, p + 8, p + 16, p + 24, b, b + 128, b + 256,
                                         b + 384, kIdPV, i > 0 || half > 0, 1u);
                        }
                        mma_commit_warp(&pv_done[t]);
                        mma_commit_warp(&kv_empty[vslot]);
                    } else if (lane == 0) {
                        mbar_arrive(&kv_empty[vslot]);
                    }
                    if (more) {
                        if (i + 1 < e) {
                            S();
                            mma_commit_warp(&s_full[t]);
                            mma_commit_warp(&kv_empty[slot]);
                            if (i + 2 == e) mma_commit_warp(&q_empty[t]);  // the last S is issued
                        } else if (lane == 0) {
                            mbar_arrive(&kv_empty[slot]);
                        }
                        next();
                    }
                    pass_turn();
                }
            }
            // completes once every MMA that this warp issued has finished
            mma_commit_warp(&all_done[t]);
            if (lane == 0) wait_plain(&all_done[t], 0, a.limit);
            __syncwarp();
        }
    } else {
        reg_alloc<kRegsMany>();
        // ---------------- softmax: thread = row ----------------
        const int t = (warp - 4) >> 2;
        const int wq = warp & 3;
        const int r = wq * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t scol = tmem + lane_base + 128 * t, ocol = tmem + lane_base + 256 + 128 * t;
        const int rt = r / G, rh = r % G;  // token of the tile, head of the group
        const float c = a.c;
        uint32_t ns = 0;  // tiles this row tile has seen
        bool ok = !*abort_flag;
        for (uint32_t n = 0; ok; ++n) {
            const int us = n & 1;
            ok = __all_sync(0xffffffffu, wait_bar(&u_full[us], (n >> 1) & 1u, abort_flag, a.status, a.limit));
            if (!ok) break;
            const volatile Unit &u = units[us];
            if (!u.valid) break;
            const int et = u.e[t];
            const int tok = u.tok0 + t * tpt + rt;
            const bool real = rt < tpt && tok < u.Lq;
            int left, left0;  // last key of this row, and of the tile's first one, from the tile's first key
            {
                const int Lk = u.Lk, j0 = u.j0, last = tok - rt + Lk - u.Lq;
                left = (a.causal ? min(Lk - 1, last + rt) : Lk - 1) - j0 * kTileKeys;
                // the first row keeps the fewest: key tiles that pass it are masked
                left0 = (a.causal ? min(Lk - 1, last) : Lk - 1) - j0 * kTileKeys;
            }
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < et; ++i, ++ns, left -= kTileKeys, left0 -= kTileKeys) {
                ok = wait_bar(&s_full[t], ns & 1u, abort_flag, a.status, a.limit) && ok;
                tc_fence_after();
                const uint64_t c2 = f2_pack(c, c);
                const bool masked = kTileKeys - 1 > left0;  // uniform
                bool done = false;
                if (!masked && !__any_sync(0xffffffffu, real && m == -INFINITY)) {
                    // against the reference that the row has; the loads run one part ahead
                    const uint64_t nm2 = f2_pack(-m, -m);
                    uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
                    uint32_t pk[64];
                    float s[2][32];
                    tmem_ld32(scol, s[0]);
                    tmem_wait_ld_of(s[0]);
#pragma unroll
                    for (int part = 0; part < 4; ++part) {
                        if (part < 3) tmem_ld32(scol + 32 * (part + 1), s[(part + 1) & 1]);
                        softmax_part<kPolyOf8>(s[part & 1], c2, nm2, ls2, pk + 16 * part);
                        if (part < 3) tmem_wait_ld_of(s[(part + 1) & 1]);
                    }
                    const uint64_t ls = f2_add(f2_add(ls2[0], ls2[1]), f2_add(ls2[2], ls2[3]));
                    const float sum = f2_lo(ls) + f2_hi(ls);
                    // (not >: a NaN takes the other path too)
                    done = !__any_sync(0xffffffffu, real && !(sum <= kMaxSum));
                    if (done) {
                        l += sum;
                        tmem_st32(scol, reinterpret_cast<float *>(pk));
                        tmem_st32(scol + 32, reinterpret_cast<float *>(pk + 32));
                    }
                }
                if (!done) {
                    // first, masked and exceptional tiles: the row's true maximum becomes its reference
                    float s[128];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(scol + 32 * q, s + 32 * q);
                    tmem_wait_ld();
                    if (masked) {
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
                    const float mnew = fmaxf(m, tmax);
                    // warp-uniform decision: the TMEM accesses below are collective
                    if (__any_sync(0xffffffffu, mnew > m)) {
                        const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - mnew);
                        if (i > 0) {
                            ok = wait_bar(&pv_done[t], (ns - 1) & 1u, abort_flag, a.status, a.limit) && ok;
                            tc_fence_after();
#pragma unroll
                            for (int part = 0; part < D / 16; ++part) {
                                float ov[16];
                                tmem_ld16(ocol + 16 * part, ov);
                                tmem_wait_ld();
#pragma unroll
                                for (int q = 0; q < 16; ++q) ov[q] *= alpha;
                                tmem_st16(ocol + 16 * part, reinterpret_cast<uint32_t *>(ov));
                            }
                        }
                        l *= alpha;
                        m = mnew;
                    }
                    const float mref = m == -INFINITY ? 0.f : m;  // rows without a key so far
                    const uint64_t nm2 = f2_pack(-mref, -mref);
                    uint64_t ls2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int part = 0; part < 4; ++part) {
                        uint32_t pk[16];
                        // masked scores are -inf: exactly 0 by the SFU, 2^-126 by the polynomial
                        softmax_part<0>(s + 32 * part, c2, nm2, ls2, pk);
                        tmem_st16(scol + 16 * part, pk);
                    }
                    const uint64_t ls = f2_add(f2_add(ls2[0], ls2[1]), f2_add(ls2[2], ls2[3]));
                    l += f2_lo(ls) + f2_hi(ls);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            }
            // ---------------- epilogue ----------------
            if (et > 0) ok = wait_bar(&pv_done[t], (ns - 1) & 1u, abort_flag, a.status, a.limit) && ok;
            tc_fence_after();
            ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
            if (!ok) break;
            const int head = u.hk * G + rh;
            const int64_t grow = u.q0 + tok;
            if (a.splits == 1) {
                if (real && a.lse != nullptr)
                    a.lse[head * a.total_q + grow] = l > 0.f ? (m + log2f(l)) * kFwdLn2 : l == 0.f ? -INFINITY : l;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                __nv_bfloat16 *dst = a.o.row(grow, head);
#pragma unroll
                for (int part = 0; part < D / 32; ++part) {
                    float ov[32];
                    if (et > 0) {
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
                    }
                    if (et == 0 || l == 0.f) {
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
                const int64_t slots = a.total_q * a.heads, slot = u.split * slots + grow * a.heads + head;
                if (real) reinterpret_cast<float2 *>(a.part + a.splits * slots * D)[slot] = make_float2(m, l);
#pragma unroll
                for (int part = 0; part < D / 32; ++part) {
                    float ov[32];
                    if (et > 0) {
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q) ov[q] = 0.f;
                    }
                    if (real) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<float4 *>(a.part + slot * D + 32 * part + q) =
                                make_float4(ov[q], ov[q + 1], ov[q + 2], ov[q + 3]);
                    }
                }
            }
            tc_fence_before();  // O is read: the next unit's first PV may overwrite it
            __syncwarp();
            if (lane == 0) mbar_arrive(&u_empty[us]);
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
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ Args a) {
    const int splits = a.splits;
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
                          int D, int rows, int box_heads) {
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
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(rows)};
    const cuuint32_t es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.p, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static cudaError_t launch_packed_fwd(const nabla::packed::Args &a, int64_t units, cudaStream_t stream) {
    using namespace nabla::packed;
    CUtensorMap mq, mk, mv;
    // without any key nothing is loaded; the maps only have to be valid
    const bool keys = a.total_k > 0;
    if (!nabla_make_tmap_view(&mq, a.q, a.total_q, a.heads, D, a.tile_tokens, a.group) ||
        !nabla_make_tmap_view(&mk, keys ? a.k : a.q, keys ? a.total_k : 1, keys ? a.heads_kv : 1, D, 128, 1) ||
        !nabla_make_tmap_view(&mv, keys ? a.v : a.q, keys ? a.total_k : 1, keys ? a.heads_kv : 1, D, 128, 1))
        return cudaErrorInvalidValue;
    constexpr uint32_t kSmem = FwdLayout<D>::kSmem;
    cudaError_t err = cudaFuncSetAttribute(fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           static_cast<int>(kSmem));
    if (err != cudaSuccess) return err;
    const unsigned grid = static_cast<unsigned>(units < kSms ? units : kSms);
    fwd_kernel<D><<<grid, kFwdThreads, kSmem, stream>>>(mq, mk, mv, a);
    err = cudaGetLastError();
    if (err != cudaSuccess || a.splits == 1) return err;
    const int64_t rows = a.total_q * a.heads;
    combine_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

// units: row tile pairs (an upper bound over the sequences) x heads_kv x splits
cudaError_t nabla_launch_packed_fwd(const nabla::packed::Args &a, int D, int64_t units,
                                    cudaStream_t stream) {
    return D == 128 ? launch_packed_fwd<128>(a, units, stream) : launch_packed_fwd<64>(a, units, stream);
}
