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
//   P_t = exp2(S_t scale log2e - m)   two softmax warpgroups per row tile:
//                      thread (h, r) takes row r and keys [64 h, +64)
//   O_t += P_t . V     (P_t in TMEM over S_t, V from shared memory)
// The tensor core works for one row tile while the other is in its softmax.
//
// At D = 128 a tile costs the tensor core 1,024 cycles and its 16,384
// exponentials the SFU another 1,024 (16 a cycle and SM), so part of them is
// taken on the FMA pipe instead: 2^x = 2^n p(x - n), n the nearest integer, p
// the degree-4 polynomial that minimises the largest relative error of 2^f on
// [-1/2, 1/2] (2.6e-6, found with a Remez iteration; P is rounded to bf16, by up to
// 2^-8, next).
//
// A row's reference is the maximum of its first tile (and of masked ones).
// Other tiles are taken against it without looking for their own maximum: P
// (bf16) and the float32 accumulators have the exponent range for scores far
// above it.  That leaves five instructions a pair of scores in the loop, no
// exchange between threads, and P goes over to the tensor core in two parts as
// it is made.  A unit in which some tile's sum passed 2^60 (or is NaN), or whose O
// left float32, is taken once more, moving to the true maximum at every tile.
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
// Warp roles (640 threads): warp 0 takes units and loads by TMA, warps 1 and 2
// issue the MMAs of row tiles 0 and 1, warps 4-11 and 12-19 are their softmax
// (warp 3 only completes the first warpgroup).  With one thread per row of 128
// scores there was one softmax warp of a tile on each scheduler, and its
// latencies, not its pipes, set the pace (1,450 cycles a tile).  The issuing warps stay converged
// and send four MMAs per elect.sync (a lone lane takes about as long to issue an
// MMA as it runs).  They take turns, PV_0 S_0 then PV_1 S_1, each waiting for its
// operands before its turn: the MMAs of a turn go out in one run, and the row
// tiles stay half a period apart (free-running issuers fell into step, both
// in their softmax and then both at the tensor core, and lost 15%).
// TMEM columns: S_0 [0,128), S_1 [128,256), O_0 [256, +D), O_1 [384, +D); the
// bf16 P of keys [64 h, +64) takes the first 32 columns of their scores.
#include "packed.cuh"

namespace nabla {
namespace packed {

using namespace sm100;

constexpr int kFwdThreads = 640;
// Registers a thread: the launch gives 96 to each of the five warpgroups; the
// first (loads, MMA issue) hands some over to the four softmax ones:
// 64 + 4 * 104 = 480 = 5 * 96.
constexpr int kRegsFew = 64, kRegsMany = 104;
constexpr int kTileKeys = 128;
constexpr float kFwdLn2 = 0.6931471805599453f;
constexpr float kMaxSum = 1152921504606846976.f;  // 2^60: largest sum of P over a tile's half row
// pairs of every 8 whose exponentials the FMA pipe takes.  8,192 dense tokens, 40/8
// heads, D = 128: 1 of 8 1,364 TFLOP/s, 2 1,372, 3 1,331; D = 64, where the tensor core
// has half the work and instruction issue is short: 0 and 1 alike, 2 2% and 3 6% slower.
template <int D>
constexpr int kPolyOf8 = D == 128 ? 2 : 1;

// One unit, as the loading warp hands it to the others.
struct Unit {
    int valid, hk, split;
    int exact;    // every tile moves to its true maximum
    int redo;     // set by the softmax: to be taken again, exactly
    int q0, Lq, k0, Lk;
    int tok0;     // first token of row tile 0
    int j0;       // first key tile of this split
    int e[2];     // key tiles of each row tile in it
};

template <int D>
struct FwdLayout {
    static constexpr int kHalves = D / 64;
    static constexpr int kRing = D == 128 ? 4 : 8;  // K and V tiles in flight (5 at D = 128 were no faster)
    static constexpr uint32_t kTile = 128u * D * 2;  // 128 rows x D bf16
    static constexpr uint32_t OFF_Q = 0;             // two row tiles
    static constexpr uint32_t OFF_RING = 2 * kTile;
    static constexpr uint32_t OFF_STAGE = OFF_RING + kRing * kTile;  // 2 KB per softmax warp
    static constexpr uint32_t OFF_BAR = OFF_STAGE + 16 * 2048;
    static constexpr int kBars = 2 * kRing + 4 + 2 + 4 + 2 + 4 + 1 + 4;
    static constexpr uint32_t OFF_UNIT = OFF_BAR + 8 * kBars;
    static constexpr uint32_t OFF_RED = (OFF_UNIT + 2 * sizeof(Unit) + 15) / 16 * 16;  // maxima or sums: [tile][half][row]
    static constexpr uint32_t OFF_INT = OFF_RED + 2 * 2 * 128 * 4;
    static constexpr uint32_t kSmem = OFF_INT + 16;  // (no alignment pad: aligned as declared)
};

// 2^x of a pair on the SFU
__device__ __forceinline__ uint64_t exp2_sfu(uint64_t x) {
    uint64_t y;
    asm("{\n .reg .f32 a, b;\n mov.b64 {a, b}, %1;\n ex2.approx.ftz.f32 a, a;\n ex2.approx.ftz.f32 b, b;\n"
        " mov.b64 %0, {a, b};\n}\n"
        : "=l"(y)
        : "l"(x));
    return y;
}
// x between lo and hi; a NaN stays one
__device__ __forceinline__ float clamp_nan(float x, float lo, float hi) {
    float d;
    asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, %2;\n min.NaN.f32 %0, t, %3;\n}\n" : "=f"(d) : "f"(x), "f"(lo), "f"(hi));
    return d;
}
// 2^x of a pair on the FMA pipe, for x in [-126, 126]; what lies outside is taken as
// the border.  The integer part is added to the exponent, which without the upper
// border runs into the sign and past it from 129 on.  2^126 is above kMaxSum, and so
// is what a NaN gives (0x7fffffff twice, the second shifted: the largest float32), so
// that the row's sum tells of both.  (The upper border and the NaN cost 1.3% of the
// dense and of the causal call at 8,192 tokens, D = 128; a maximum of the inputs beside
// them, looked at once a unit, cost 3-5%.)
__device__ __forceinline__ uint64_t exp2_poly(uint64_t x) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    x = f2_pack(clamp_nan(f2_lo(x), -126.f, 126.f), clamp_nan(f2_hi(x), -126.f, 126.f));
    const uint64_t t = f2_add(x, f2_pack(kRound, kRound));
    const uint64_t f = f2_fma(f2_add(t, f2_pack(-kRound, -kRound)), f2_pack(-1.f, -1.f), x);
    uint64_t p = f2_fma(f2_pack(0.009570101911165427f, 0.009570101911165427f), f,
                        f2_pack(0.055917860319388245f, 0.055917860319388245f));
    p = f2_fma(p, f, f2_pack(0.2402474482786378f, 0.2402474482786378f));
    p = f2_fma(p, f, f2_pack(0.6931218147366892f, 0.6931218147366892f));
    p = f2_fma(p, f, f2_pack(0.9999992614457122f, 0.9999992614457122f));
    // the integer stands in the low bits of t: into the exponent
    const uint32_t lo = static_cast<uint32_t>(p) + (static_cast<uint32_t>(t) << 23);
    const uint32_t hi = static_cast<uint32_t>(p >> 32) + (static_cast<uint32_t>(t >> 32) << 23);
    return f2_pack(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t pack_bf16_pair(uint64_t p) {
    uint32_t d;
    asm("{\n .reg .f32 a, b;\n mov.b64 {a, b}, %1;\n cvt.rn.bf16x2.f32 %0, b, a;\n}\n" : "=r"(d) : "l"(p));
    return d;
}

// P of 32 keys from their scores, as packed bf16; adds the values to two pairs of sums.
template <int kPoly>
__device__ __forceinline__ void softmax_part(const float *s, uint64_t c2, uint64_t nm2,
                                             uint64_t *ls2, uint32_t *pk) {
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        const uint64_t x = f2_fma(f2_pack(s[k], s[k + 1]), c2, nm2);
        // the polynomial's pairs are spread over the row, so that both pipes are busy at once
        const bool poly = ((k >> 1) * kPoly) % 8 + kPoly > 7 && kPoly > 0;
        const uint64_t p = poly ? exp2_poly(x) : exp2_sfu(x);
        ls2[(k >> 1) & 1] = f2_add(ls2[(k >> 1) & 1], p);
        pk[k >> 1] = pack_bf16_pair(p);
    }
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, const __grid_constant__ Args a) {
    using L = FwdLayout<D>;
    constexpr int kRing = L::kRing, kHalves = L::kHalves;
    constexpr uint32_t kTile = L::kTile;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t sb = smem_addr(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + L::OFF_BAR);
    uint64_t *kv_full = bar, *kv_empty = bar + kRing;
    uint64_t *q_full = bar + 2 * kRing, *q_empty = q_full + 2;  // per row tile
    // per row tile: S complete; the two parts of P written (its eight warps); PV complete
    uint64_t *s_full = q_empty + 2, *p_full = s_full + 2, *pv_done = p_full + 4;
    // per unit slot: written by the loading warp; read by the 18 others
    uint64_t *u_full = pv_done + 2, *u_empty = u_full + 2;
    uint64_t *raw_full = u_empty + 2;  // a tile that still has rows to zero
    uint64_t *all_done = raw_full + 1, *turn = all_done + 2;  // per issuing warp
    volatile Unit *units = reinterpret_cast<Unit *>(sm + L::OFF_UNIT);
    int *sInt = reinterpret_cast<int *>(sm + L::OFF_INT);  // [0] tmem base [2] abort
    volatile int *abort_flag = sInt + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.group, tpt = a.tile_tokens;  // tokens a row tile

    allow_dependents();  // combine_kernel, up to its wait
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
            mbar_init(&p_full[2 * t], 8);
            mbar_init(&p_full[2 * t + 1], 8);
            mbar_init(&pv_done[t], 1);
            mbar_init(&u_full[t], 1);
            mbar_init(&u_empty[t], 18);
        }
        mbar_init(raw_full, 1);
        sInt[2] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(&sInt[0]), 512);
        tmem_relinquish();
    }
    // every CTA looks at every border before anything is written
    const bool good = borders_ok(a, threadIdx.x, kFwdThreads) && (sb & 1023u) == 0;  // (swizzled tiles need the alignment asked for above)
    tc_fence_before();
    const bool go = !__syncthreads_or(!good);
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(sInt[0]);
    // (all CTAs see the same borders; a wait that expires is a second away)
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicExch(a.status, go ? kDevOk : kDevParam);
    if (!go) {
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
            int64_t x = blockIdx.x;  // the first unit; the counter hands out those behind the grid's
            for (uint32_t n = 0; ok; ++n) {
                // the slot's last unit is finished: it may have to be taken again
                const int us = n & 1;
                ok = __all_sync(0xffffffffu, lane != 0 || wait_bar(&u_empty[us], ((n >> 1) & 1u) ^ 1u, abort_flag,
                                                                   a.status, a.limit));
                if (!ok) break;
                Unit u = {};
                int again = n >= 2 && units[us].redo != 0 ? us : -1;
                if (again < 0) {
                    x = __shfl_sync(0xffffffffu, x, 0);
                    const int64_t now = x;
                    if (now < a.units) {
                        // the next one, under this one's loads
                        if (lane == 0) x = a.units > gridDim.x ? take_unit(a) : a.units;
                        const int64_t ux = now / a.splits;
                        SeqTile st;
                        u.split = static_cast<int>(now % a.splits);
                        u.hk = static_cast<int>(ux % a.heads_kv);
                        u.valid = scan.find(a, ux / a.heads_kv, 1, 2 * tpt, lane, &st);
                        if (u.valid) {
                            u.q0 = st.q0;
                            u.Lq = st.Lq;
                            u.k0 = st.k0;
                            u.Lk = st.Lk;
                            // the last tiles of a causal sequence keep the most keys: they go first
                            u.tok0 = ((u.Lq + 2 * tpt - 1) / (2 * tpt) - 1 - st.tile) * 2 * tpt;
                        }
                    }
                    if (!u.valid && n >= 1) {  // the end, unless the other slot's unit has to be taken again
                        ok = __all_sync(0xffffffffu, lane != 0 || wait_bar(&u_empty[us ^ 1], ((n - 1) >> 1) & 1u,
                                                                           abort_flag, a.status, a.limit));
                        if (!ok) break;
                        if (units[us ^ 1].redo != 0) again = us ^ 1;
                    }
                }
                if (again >= 0) {
                    volatile Unit &w = units[again];
                    u.valid = u.exact = 1;
                    u.hk = w.hk;
                    u.split = w.split;
                    u.q0 = w.q0;
                    u.Lq = w.Lq;
                    u.k0 = w.k0;
                    u.Lk = w.Lk;
                    u.tok0 = w.tok0;
                    u.j0 = w.j0;
                    u.e[0] = w.e[0];
                    u.e[1] = w.e[1];
                    __syncwarp();
                    if (lane == 0) w.redo = 0;
                } else if (u.valid) {
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
                }
                const int emax = max(u.e[0], u.e[1]);
                __syncwarp();
                if (lane == 0) {
                    volatile Unit &w = units[us];
                    w.valid = u.valid;
                    w.exact = u.exact;
                    w.redo = 0;
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
                if (!ok || a.stall) break;
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
            // at D = 128 the turn passes in front of the last four MMAs, whose run hides
            // the change (1,257 against 1,240 TFLOP/s); at D = 64 there are only four,
            // and passing in front of them lost 7%
            auto S = [&]() {
                const uint64_t kd = desc_sw128(sb + L::OFF_RING + slot * kTile, 16, 1024);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    if (h == 1) pass_turn();
                    const uint32_t o = h * 1024;  // halves 16 KB, 16 features 32 bytes
                    mma_ss4_warp(ds, ds, ds, ds, qd + o, qd + o + 2, qd + o + 4, qd + o + 6, kd + o, kd + o + 2,
                                 kd + o + 4, kd + o + 6, kIdS, h > 0, 1u);
                }
                if (kHalves == 1) pass_turn();
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
                // turn -1: S(0); turn i: PV(i), S(i + 1).  The waits of a turn stand in
                // front of it, but for the second part of P, made under the first's MMAs.
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
                } else {
                    if (lane == 0) mbar_arrive(&kv_empty[slot]);
                    pass_turn();
                }
                next();
                for (int i = 0; ok && i < emax; ++i) {
                    const bool more = i + 1 < emax;
                    ok = arrived();  // V(i)
                    const uint32_t vslot = slot;
                    next();
                    if (ok && more) ok = arrived();  // K(i + 1)
                    if (ok && i < e) ok = warp_wait(&p_full[2 * t], np & 1u, abort_flag, a.status, a.limit);
                    ok = ok && my_turn();
                    if (!ok) break;
                    tc_fence_after();
                    if (i < e) {
                        const uint64_t vd = desc_sw128(sb + L::OFF_RING + vslot * kTile, 16384, 1024);
                        // part p of P: keys [32 p, +32) and [64 + 32 p, +32); 16 keys are 8
                        // columns of P and 2 KB of V
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            if (part == 1) {
                                ok = warp_wait(&p_full[2 * t + 1], np & 1u, abort_flag, a.status, a.limit);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            const uint32_t p = ds + 16 * part;
                            const uint64_t b = vd + 256 * part;
                            mma_ts4_warp(dov, dov, dov, dov, p, p + 8, p + 64, p + 72, b, b + 128, b + 512,
                                         b + 640, kIdPV, i > 0 || part > 0, 1u);
                        }
                        if (!ok) break;
                        ++np;
                        mma_commit_warp(&pv_done[t]);
                        mma_commit_warp(&kv_empty[vslot]);
                    } else if (lane == 0) {
                        mbar_arrive(&kv_empty[vslot]);
                    }
                    if (i + 1 >= e) pass_turn();
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
                }
            }
            // completes once every MMA that this warp issued has finished
            mma_commit_warp(&all_done[t]);
            if (lane == 0) wait_plain(&all_done[t], 0, a.limit);
            __syncwarp();
        }
    } else {
        reg_alloc<kRegsMany>();
        // ---------------- softmax: row r of row tile t, keys [64 h, +64) of each key tile ----------------
        const int t = (warp - 4) >> 3, h = ((warp - 4) >> 2) & 1;
        const int wq = warp & 3;
        const int r = wq * 32 + lane;
        const int pair = 1 + 4 * t + wq;  // named barrier of the two warps that share rows
        float *red = reinterpret_cast<float *>(sm + L::OFF_RED) + t * 256 + r;  // this row's maxima, then sums
        const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t scol = tmem + lane_base + 128 * t + 64 * h;
        const uint32_t ocol = tmem + lane_base + 256 + 128 * t + (D / 2) * h;  // this half's share of O
        const int rt = r / G, rh = r % G;  // token of the tile, head of the group
        const float c = a.c;
        const uint64_t c2 = f2_pack(c, c);
        uint32_t ns = 0;  // tiles this row tile has seen
        bool ok = true;
        // The two warps that share rows meet at named barriers, so they go on or give
        // up together.
        auto both = [&](bool good) -> bool { return !bar_or(pair, 64, !good || *abort_flag != 0); };
        for (uint32_t n = 0; ok; ++n) {
            const int us = n & 1;
            ok = both(wait_bar(&u_full[us], (n >> 1) & 1u, abort_flag, a.status, a.limit));
            if (!ok) break;
            const volatile Unit &u = units[us];
            if (!u.valid) break;
            const int et = u.e[t];
            const int tok = u.tok0 + t * tpt + rt;
            const bool real = rt < tpt && tok >= 0 && tok < u.Lq;
            int left, left0;  // last key of this row, and of the tile's first one, from this half's first key
            {
                const int Lk = u.Lk, first = u.j0 * kTileKeys + 64 * h, last = tok - rt + Lk - u.Lq;
                left = (a.causal ? min(Lk - 1, last + rt) : Lk - 1) - first;
                // the first row keeps the fewest: key tiles that pass it are masked (both halves)
                left0 = (a.causal ? min(Lk - 1, last) : Lk - 1) - u.j0 * kTileKeys;
            }
            float m = -INFINITY, l = 0.f;  // m is the same in both halves
            const bool exact = u.exact != 0;
            bool over = false;
            for (int i = 0; i < et; ++i, ++ns, left -= kTileKeys, left0 -= kTileKeys) {
                ok = wait_bar(&s_full[t], ns & 1u, abort_flag, a.status, a.limit) && ok;
                tc_fence_after();
                const bool masked = kTileKeys - 1 > left0;  // uniform over the tile
                auto hand_over = [&](int part) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + part]);
                };
                uint64_t ls2[2] = {0ull, 0ull};
                if (i > 0 && !masked && !exact) {
                    const uint64_t nm2 = f2_pack(-m, -m);  // (m is a number: the first tile was not masked)
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        float s[32];
                        uint32_t pk[16];
                        tmem_ld32(scol + 32 * part, s);
                        tmem_wait_ld_of(s);
                        softmax_part<kPolyOf8<D>>(s, c2, nm2, ls2, pk);
                        tmem_st16(scol + 16 * part, pk);
                        hand_over(part);
                    }
                    const uint64_t ls = f2_add(ls2[0], ls2[1]);
                    const float sum = f2_lo(ls) + f2_hi(ls);
                    over |= real && !(sum <= kMaxSum);  // (not >: a NaN counts)
                    l += sum;
                } else {
                    // first, masked and exact tiles: the row's true maximum becomes its reference
                    float s[32];
                    auto scores = [&](int part) {
                        tmem_ld32(scol + 32 * part, s);
                        tmem_wait_ld_of(s);
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) s[k] = 32 * part + k <= left ? s[k] : -INFINITY;
                        }
                    };
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        scores(part);
#pragma unroll
                        for (int k = 0; k < 32; k += 2) mx[(k >> 1) & 3] = fmax3(mx[(k >> 1) & 3], s[k], s[k + 1]);
                    }
                    const float tmax = c * fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
                    red[128 * h] = tmax;
                    bar_sync(pair, 64);
                    const float mnew = fmax3(m, tmax, red[128 * (h ^ 1)]);
                    // uniform over both warps' rows: the TMEM accesses below are collective
                    if (__any_sync(0xffffffffu, mnew > m)) {
                        const float alpha = m == -INFINITY ? 0.f : fast_exp2(m - mnew);
                        if (i > 0) {
                            ok = wait_bar(&pv_done[t], (ns - 1) & 1u, abort_flag, a.status, a.limit) && ok;
                            tc_fence_after();
#pragma unroll
                            for (int part = 0; part < D / 32; ++part) {
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
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t pk[16];
                        scores(part);  // (their P goes over scores that were read before)
                        // masked scores are -inf: exactly 0 by the SFU, 2^-126 by the polynomial
                        softmax_part<0>(s, c2, nm2, ls2, pk);
                        tmem_st16(scol + 16 * part, pk);
                        hand_over(part);
                    }
                    const uint64_t ls = f2_add(ls2[0], ls2[1]);
                    l += f2_lo(ls) + f2_hi(ls);
                }
            }
            // ---------------- epilogue: half h writes features [D/2 h, +D/2) ----------------
            bool again = false;
            if (et > 0) {
                ok = wait_bar(&pv_done[t], (ns - 1) & 1u, abort_flag, a.status, a.limit) && ok;
                red[128 * h] = l;
                again = bar_or(pair, 64, over);  // (and the sums are exchanged)
                l += red[128 * (h ^ 1)];
                if (again && lane == 0) units[us].redo = 1;
            }
            tc_fence_after();
            ok = both(ok);  // (and the sums are read before the next unit's maxima)
            if (!ok) break;
            const int head = u.hk * G + rh;
            const int64_t grow = u.q0 + tok;
            // P up to 2^60 times a large v may have left float32 where the row does not: such a
            // unit is taken again as well (what is written now is written over).  Costs 0.7% of
            // causal prompts and 1.2% of the dense call at 8,192 tokens, D = 128, in registers
            // more than in time; with one vote behind both parts it was 1.2% and 2%.
            auto finite = [&](const float *ov) {
                float big = 0.f;
#pragma unroll
                for (int q = 0; q < 32; q += 2)
                    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(big) : "f"(fabsf(ov[q])), "f"(fabsf(ov[q + 1])));
                if (real && !exact && !(big < INFINITY)) units[us].redo = 1;
            };
            if (again) {
                // nothing of these rows is written this time
            } else if (a.splits == 1) {
                if (h == 0 && real && a.lse != nullptr)
                    a.lse[head * a.total_q + grow] = l > 0.f ? (m + log2f(l)) * kFwdLn2 : l == 0.f ? -INFINITY : l;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                __nv_bfloat16 *dst = real ? a.o.row(grow, head) + (D / 2) * h : nullptr;
                unsigned char *stage = sm + L::OFF_STAGE + (warp - 4) * 2048;
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    float ov[32];
                    if (et > 0) {
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
                        finite(ov);
                    }
                    if (et == 0 || l == 0.f) {
#pragma unroll
                        for (int q = 0; q < 32; ++q) ov[q] = 0.f;
                    }
                    uint4 w[4];
#pragma unroll
                    for (int e8 = 0; e8 < 4; ++e8) {
                        w[e8].x = pack_bf16(ov[8 * e8] * inv, ov[8 * e8 + 1] * inv);
                        w[e8].y = pack_bf16(ov[8 * e8 + 2] * inv, ov[8 * e8 + 3] * inv);
                        w[e8].z = pack_bf16(ov[8 * e8 + 4] * inv, ov[8 * e8 + 5] * inv);
                        w[e8].w = pack_bf16(ov[8 * e8 + 6] * inv, ov[8 * e8 + 7] * inv);
                    }
                    store_rows(stage, w, dst == nullptr ? nullptr : dst + 32 * part, lane);
                }
            } else {
                // unnormalised part of this split: [split][token][head][D], then (m, l)
                const int64_t slots = a.total_q * a.heads, slot = u.split * slots + grow * a.heads + head;
                if (h == 0 && real)
                    reinterpret_cast<float2 *>(a.part + a.splits * slots * D)[slot] = make_float2(m, l);
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    float ov[32];
                    if (et > 0) {
                        tmem_ld32(ocol + 32 * part, ov);
                        tmem_wait_ld();
                        finite(ov);
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q) ov[q] = 0.f;
                    }
                    if (real) {
#pragma unroll
                        for (int q = 0; q < 32; q += 4)
                            *reinterpret_cast<float4 *>(a.part + slot * D + (D / 2) * h + 32 * part + q) =
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
    wait_for_prerequisites();
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
static cudaError_t launch_packed_fwd(const nabla::packed::Args &a, cudaStream_t stream) {
    using namespace nabla::packed;
    CUtensorMap mq, mk, mv;
    // without any key nothing is loaded; the maps only have to be valid
    const bool keys = a.total_k > 0;
    if (!nabla_make_tmap_view(&mq, a.q, a.total_q, a.heads, D, a.tile_tokens, a.group) ||
        !nabla_make_tmap_view(&mk, keys ? a.k : a.q, keys ? a.total_k : 1, keys ? a.heads_kv : 1, D, 128, 1) ||
        !nabla_make_tmap_view(&mv, keys ? a.v : a.q, keys ? a.total_k : 1, keys ? a.heads_kv : 1, D, 128, 1))
        return cudaErrorInvalidValue;
    constexpr uint32_t kSmem = FwdLayout<D>::kSmem;
    cudaError_t err = nabla_allow_smem<fwd_kernel<D>>(kSmem);
    if (err != cudaSuccess) return err;
    const unsigned grid = static_cast<unsigned>(a.units < kSms ? a.units : kSms);
    fwd_kernel<D><<<grid, kFwdThreads, kSmem, stream>>>(mq, mk, mv, a);
    err = cudaGetLastError();
    if (err != cudaSuccess || a.splits == 1) return err;
    const int64_t rows = a.total_q * a.heads;
    return nabla_launch_early(combine_kernel<D>, static_cast<unsigned>((rows + 7) / 8), 256, 0, stream, a);
}

cudaError_t nabla_launch_packed_fwd(const nabla::packed::Args &a, int D, cudaStream_t stream) {
    return D == 128 ? launch_packed_fwd<128>(a, stream) : launch_packed_fwd<64>(a, stream);
}
