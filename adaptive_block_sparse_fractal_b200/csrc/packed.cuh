// Shared by the packed-sequence attention kernels (packed_fwd.cu,
// packed_bwd.cu): their arguments, the search for a CTA's sequence, and the
// tensor maps over strided [tokens, heads, D] views.
#pragma once

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
    int *status;       // workspace status word
    float *pad_l, *pad_d;  // backward: [heads, pad_rows], -lse log2(e) and -dout.o
    float *part;       // split forward: partial rows, then their (m, l)
    int64_t total_q, total_k, pad_rows;
    int seqs, heads, heads_kv, group, causal;
    float c, scale;    // scale * log2(e), scale
    uint32_t limit;    // ns per wait
};

struct SeqTile {
    int seq, tile;      // tile within the sequence
    int q0, Lq, k0, Lk;
    int pad;            // 64-row tiles of the sequences in front
};

// Finds the sequence that holds tile `unit`, sequences having `count(Lq, Lk)`
// tiles each, by a scan of all threads of the CTA (NT of them) over the
// borders.  Every CTA looks at every border: one that does not ascend or
// leaves the tensors makes all of them give up before any output is written.
// Returns false when the CTA has nothing to do.
template <int NT, typename Count>
__device__ __forceinline__ bool find_seq(const Args &a, int64_t unit, Count count, SeqTile *out,
                                         int64_t *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = NT / 32;
    int64_t carry = 0;  // low half: tiles, high half: 64-row tiles of q
    if (threadIdx.x == 0) out->seq = -1;
    bool bad = false;
    for (int base = 0; base < a.seqs; base += NT) {
        const int s = base + threadIdx.x;
        int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
        if (s < a.seqs) {
            q0 = a.cu_q[s];
            q1 = a.cu_q[s + 1];
            k0 = a.cu_k[s];
            k1 = a.cu_k[s + 1];
        }
        bad |= q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k;
        const int64_t n = bad ? 0 : count(q1 - q0, k1 - k0);
        const int64_t mine = n | (static_cast<int64_t>(bad ? 0 : (q1 - q0 + 63) >> 6) << 32);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();  // the sums of the round before have been read
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        int64_t front = carry, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) front += warp_sums[w];
            all += warp_sums[w];
        }
        carry += all;
        const int64_t excl = front + incl - mine;
        const int64_t before = excl & 0xffffffffll;
        if (unit >= before && unit < before + n) {
            out->seq = s;
            out->tile = static_cast<int>(unit - before);
            out->q0 = q0;
            out->Lq = q1 - q0;
            out->k0 = k0;
            out->Lk = k1 - k0;
            out->pad = static_cast<int>(excl >> 32);
        }
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicExch(a.status, kDevParam);
        return false;
    }
    return out->seq >= 0;
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

// Host: tensor map over a [tokens, heads, D] bf16 view, boxes of 64 features of
// one head x `rows` tokens, 128-byte swizzle (defined in packed_fwd.cu).
bool nabla_make_tmap_view(CUtensorMap *m, const nabla::packed::View &v, int64_t tokens, int heads,
                          int D, int rows);
