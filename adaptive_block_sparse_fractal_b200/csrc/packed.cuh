// Shared by the packed-sequence attention kernels (packed_fwd.cu,
// packed_bwd.cu): their arguments, the search for a CTA's sequence, and the
// tensor maps over strided [tokens, heads, D] views.
#pragma once

#include "launch.cuh"
#include "sm100.cuh"

namespace nabla {
namespace packed {

struct View {  // bf16 [tokens, heads, D], distances in elements
    __nv_bfloat16 *p;
    int64_t token, head;
    __device__ __forceinline__ __nv_bfloat16 *row(int64_t t, int h) const {
        return p + t * token + h * head;
    }
};

struct Args {
    View q, k, v, o, dout, dq, dk, dv;
    const int32_t *cu_q, *cu_k;
    float *lse;        // [heads, total_q]
    int *status;       // workspace status word; behind it the unit counter and, in the backward, whether borders are bad
    float *pad_l, *pad_d;  // backward: [heads, pad_rows], -lse log2(e) and -dout.o
    float *part;       // split forward: partial rows, then their (m, l)
    int64_t total_q, total_k, pad_rows;
    uint32_t units;    // of a persistent launch, at most
    int seqs, heads, heads_kv, group, causal;
    int tile_tokens, splits;  // forward: tokens a row tile (128 / group), splits of the key range
    float c, scale;    // scale * log2(e), scale
    uint32_t limit;    // ns per wait
    int stall;         // test aid: no keys (dK, dV: no queries) are loaded, so that the waits for them expire
};

struct SeqTile {
    int seq, tile;      // tile within the sequence
    int q0, Lq, k0, Lk;
    int pad;            // tile_slot of its 64-row tiles of q
};

// Tiles of `len` rows are numbered so that those of sequence s begin at tile_slot(its
// first border, len, s): each sequence has room for the tiles that it may need, as
// floor((c + n) / len) + 1 >= floor(c / len) + ceil(n / len), there are total / len +
// seqs of them at most, and no sum over the sequences in front is needed.
__device__ __forceinline__ int tile_slot(int border, int len, int s) { return border / len + s; }

// Finds the sequence that holds tile `unit` of `len` rows, of q or of k: every warp
// searches by itself, 32 borders at a time (with a scan over all of them the work grew with
// the square of the sequences: 20,000 of 20 rows took 27 ms backward, against 5.3).
// Returns false when the CTA has nothing to do, be it that the borders around it are no
// borders.  For the whole CTA.
__device__ __forceinline__ bool find_seq(const Args &a, bool of_q, int len, int unit, SeqTile *out) {
    const int lane = threadIdx.x & 31;
    const int32_t *cu = of_q ? a.cu_q : a.cu_k;
    int s = 0;
    for (int n = a.seqs; n > 1;) {  // the last one of [s, s + n) that begins at or before `unit`
        const int step = (n + 31) / 32, at = lane * step;
        const uint32_t ok = __ballot_sync(0xffffffffu, at < n && tile_slot(cu[s + (at < n ? at : 0)], len, s + at) <= unit);
        const int front = ok == 0 ? 0 : (31 - __clz(ok)) * step;
        s += front;
        n = min(step, n - front);
    }
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
    const bool good = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k;
    const int tile = good ? unit - tile_slot(of_q ? q0 : k0, len, s) : -1;
    if (threadIdx.x == 0) {
        out->seq = tile >= 0 && tile < ((of_q ? q1 - q0 : k1 - k0) + len - 1) / len ? s : -1;
        out->tile = tile;
        out->q0 = q0;
        out->Lq = q1 - q0;
        out->k0 = k0;
        out->Lk = k1 - k0;
        out->pad = tile_slot(q0, 64, s);
    }
    __syncthreads();
    return out->seq >= 0;
}

constexpr int kSms = 148;  // CTAs of a persistent launch

// Borders that do not ascend or leave the tensors make a call give up before any output
// is written.  Every thread looks at some, `first` of `count` threads.
__device__ __forceinline__ bool borders_ok(const Args &a, int64_t first, int count) {
    bool good = true;
    for (int64_t s = first; s < a.seqs; s += count) {
        const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
        good = good && q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k;
    }
    return good;
}

// The next unit of a persistent launch, whose CTAs begin with the unit of their
// own index (the counter starts at 0; the order in which CTAs take units does not
// change what a unit computes).
__device__ __forceinline__ uint32_t take_unit(const Args &a) {  // (units stay below 2^31)
    return gridDim.x + atomicAdd(reinterpret_cast<unsigned int *>(a.status) + 1, 1u);
}

// One warp's walk over the sequences for units that only grow: 32 sequences at
// a time, their borders and running tile counts in registers.  A sequence has
// ceil(Lq * mul / len) tiles.
struct UnitScan {
    int base, q0, q1, k0, k1;
    uint32_t front, all;     // tiles in front of this lane's sequence and of the next 32
    __device__ __forceinline__ UnitScan() : base(-32), q0(0), q1(0), k0(0), k1(0), front(0), all(0) {}
    // sequence and tile of unit x; false behind the last
    __device__ __forceinline__ bool find(const Args &a, uint32_t x, int mul, int len, int lane, SeqTile *u) {
        while (x >= all) {
            base += 32;
            if (base >= a.seqs) {
                base -= 32;
                return false;
            }
            const int s = base + lane;
            q0 = q1 = k0 = k1 = 0;
            if (s < a.seqs) {
                q0 = a.cu_q[s];
                q1 = a.cu_q[s + 1];
                k0 = a.cu_k[s];
                k1 = a.cu_k[s + 1];
            }
            const uint32_t mine = (static_cast<uint32_t>(q1 - q0) * mul + len - 1) / len;
            uint32_t incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            front = all + incl - mine;
            all += __shfl_sync(0xffffffffu, incl, 31);
        }
        // the last lane whose sequence starts at or before x (empty ones share a start)
        const uint32_t at = __ballot_sync(0xffffffffu, front <= x);
        const int src = 31 - __clz(at);
        u->seq = base + src;
        u->q0 = __shfl_sync(0xffffffffu, q0, src);
        u->Lq = __shfl_sync(0xffffffffu, q1, src) - u->q0;
        u->k0 = __shfl_sync(0xffffffffu, k0, src);
        u->Lk = __shfl_sync(0xffffffffu, k1, src) - u->k0;
        u->pad = tile_slot(u->q0, 64, u->seq);
        u->tile = static_cast<int>(x - __shfl_sync(0xffffffffu, front, src));
        return true;
    }
};

// Rows of a warp's 32 threads -> global memory, 32 features of each: the rows
// pass through 2 KB of shared memory, so that four lanes write 64 bytes of one
// row (each thread storing its own row touches 32 rows an instruction and half
// a sector of each).  `dst` is this lane's row, null where it is not written.
__device__ __forceinline__ void store_rows(unsigned char *stage, const uint4 *w, __nv_bfloat16 *dst, int lane) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4 *>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = w[c];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = 8 * q + (lane >> 2), c = lane & 3;
        const uint4 v = *reinterpret_cast<const uint4 *>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
        const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), row);
        if (p != 0) *(reinterpret_cast<uint4 *>(p) + c) = v;
    }
    __syncwarp();
}

// box of 64 features x one head x `rows` tokens
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                            int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5}], [%2];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// 32 lanes x 16 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// tcgen05.wait::ld that the 32 values of a load pass through, so that their
// uses stay behind it while other loads or arithmetic are in flight.
__device__ __forceinline__ void tmem_wait_ld_of(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}

// Register share of a warpgroup (all four of its warps execute it).
template <int N>
__device__ __forceinline__ void reg_alloc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dealloc() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Zeroes rows [from, rows) of a tile of D features held as 64-feature halves
// of `half_bytes` each (128-byte rows, swizzled within 1024 bytes: a whole row
// is its own 128 bytes), by one warp, and makes it visible to the tensor core.
__device__ __forceinline__ void zero_rows(unsigned char *tile, int from, int rows, int halves,
                                          int half_bytes, int lane) {
    for (int h = 0; h < halves; ++h)
        for (int i = from * 8 + lane; i < rows * 8; i += 32)
            *reinterpret_cast<uint4 *>(tile + h * half_bytes + i * 16) = make_uint4(0, 0, 0, 0);
    sm100::fence_async_smem();
    __syncwarp();
}

}  // namespace packed
}  // namespace nabla

// Host: tensor map over a [tokens, heads, D] bf16 view, boxes of 64 features x
// box_heads heads x `rows` tokens, 128-byte swizzle (defined in packed_fwd.cu).
bool nabla_make_tmap_view(CUtensorMap *m, const nabla::packed::View &v, int64_t tokens, int heads,
                          int D, int rows, int box_heads);
