// Rotary positions on up to three axes, optionally fused with the fractal
// flattening of the same tensors:
//   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi),
//   phi = (pos_axis + offset) * scale * theta^(-i / pairs).
//
// HBM-bound: every element is read once and written once (2 flop a byte at
// most).  A token's angles are the same for all heads of q and k, so a thread
// owns one 16-byte chunk of the features of ONE token, takes the sine and
// cosine of its pairs once, and walks the heads of both tensors with them in
// registers; the loads of eight heads (four of two pieces each) are in flight
// before the first store.
//
// The angle is reduced in float64 (turns minus the nearest quarter turn): at
// position 1e5 a float32 angle is off by 6e-3, the float64 one by 1e-11.  The
// remainder, at most an eighth of a turn, goes to short series in float32.
#include <cuda_fp16.h>

#include "common.cuh"
#include "rope.cuh"

namespace nabla {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half &d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float &d, float v) { d = v; }

// V elements moved as one access (V * sizeof(T) = 16) or one by one.  The wide
// ones are marked as streaming: 6.4 TB/s against 5.4 TB/s at 1.6 GB each way.
template <typename T, int V>
struct alignas(V * sizeof(T) >= 16 ? 16 : alignof(T)) Frag {
    T e[V];
};

template <typename T, int V>
__device__ __forceinline__ Frag<T, V> load_frag(const T *p) {
    Frag<T, V> f;
    if constexpr (V * sizeof(T) == 16) {
        *reinterpret_cast<uint4 *>(&f) = __ldcs(reinterpret_cast<const uint4 *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f.e[i] = p[i];
    }
    return f;
}
template <typename T, int V>
__device__ __forceinline__ void store_frag(T *p, const Frag<T, V> &f) {
    if constexpr (V * sizeof(T) == 16) {
        __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&f));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = f.e[i];
    }
}

// Sine and cosine of r turns, |r| <= 1/8: Taylor series of x = 2 pi r, |x| <= pi/4,
// whose first terms left out are x^11 / 11! < 2e-9 and x^10 / 10! < 3e-8.
__device__ __forceinline__ void sincos_eighth(float r, float &s, float &c) {
    const float x = r * 6.283185307179586f, z = x * x;
    float p = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
    p = fmaf(p, z, 1.f / 120.f);
    p = fmaf(p, z, -1.f / 6.f);
    s = fmaf(p * z, x, x);
    float q = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
    q = fmaf(q, z, 1.f / 24.f);
    q = fmaf(q, z, -0.5f);
    c = fmaf(q, z, 1.f);
}

// LAYOUT 0: pairs (2i, 2i+1), a chunk is V features; 1: pairs (i, i + R), a
// chunk is V features of the first half and V of the second, then plain chunks
// of V features behind the rotated ones.
template <typename T, int LAYOUT, int V>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kPairs = LAYOUT == 0 ? V / 2 : V;
    constexpr int kFrags = LAYOUT == 0 ? 1 : 2;
    constexpr int U = V * sizeof(T) == 16 && LAYOUT == 0 ? 8 : 4;  // heads in flight
    const int tok = blockIdx.x * blockDim.y + threadIdx.y;
    if (tok >= a.N) return;
    const int b = blockIdx.z;
    const int h0 = blockIdx.y * a.heads_per_cta;
    const int c = threadIdx.x;
    const int R = a.pairs;

    // grid coordinates and the token's place on either side
    const int x = tok % a.W, ty = tok / a.W;
    const int y = ty % a.H, t = ty / a.H;
    int64_t src = tok, dst = tok;
    if (a.flat_in | a.flat_out) {
        const int P = a.P;
        const int flat = ((t * (a.H / P) + y / P) * (a.W / P) + x / P) * P * P + (y % P) * P + x % P;
        if (a.flat_in) src = flat;
        if (a.flat_out) dst = flat;
    }

    const int first = LAYOUT == 0 ? c * kPairs : c * V;  // first pair of the chunk
    const bool rotates = first < R;
    const int off0 = LAYOUT == 0 ? c * V : (rotates ? c * V : R + c * V);
    float cs[kPairs], sn[kPairs];
    if (rotates) {
        double p[3] = {t + a.offset[0], y + a.offset[1], x + a.offset[2]};
        if (a.pos != nullptr) {
            const int32_t *q = a.pos + b * a.pos_batch + static_cast<int64_t>(tok) * a.pos_axes;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                p[i] = i < a.pos_axes ? q[i] + a.offset[i] : 0.0;
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int pr = min(first + i, R - 1);
            const int ax = a.axis[pr];
            const double turns = (ax == 0 ? p[0] : ax == 1 ? p[1] : p[2]) * a.turn[pr];
            // quarter turns nearest to it (adding 1.5 * 2^52 rounds to an integer,
            // whose low bits then stand in the low word), and the rest in [-1/8, 1/8]
            const double big = fma(turns, 4.0, 6755399441055744.0);
            const float rest = static_cast<float>(fma(big - 6755399441055744.0, -0.25, turns));
            const int quad = __double2loint(big) & 3;
            float s1, c1;
            sincos_eighth(rest, s1, c1);
            const float c2 = (quad & 1) ? s1 : c1, s2 = (quad & 1) ? c1 : s1;
            cs[i] = (quad == 1 || quad == 2) ? -c2 : c2;
            sn[i] = quad >= 2 ? -s2 : s2;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) cs[i] = 1.f, sn[i] = 0.f;
    }

    const int heads = a.t[0].heads + (a.count > 1 ? a.t[1].heads : 0);
    const int h1 = min(heads, h0 + a.heads_per_cta);
    for (int hb = h0; hb < h1; hb += U) {
        Frag<T, V> f[U][kFrags];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u;
            if (h < h1) {
                const bool second = h >= a.t[0].heads;
                const RopeTensor &x = a.t[second];
                const T *p = static_cast<const T *>(x.in) + b * x.in_batch + src * x.in_token +
                             (second ? h - a.t[0].heads : h) * x.in_head + off0;
                f[u][0] = load_frag<T, V>(p);
                if (LAYOUT == 1 && rotates) f[u][kFrags - 1] = load_frag<T, V>(p + R);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u;
            if (h < h1) {
                const bool second = h >= a.t[0].heads;
                const RopeTensor &x = a.t[second];
                T *p = static_cast<T *>(x.out) + b * x.out_batch + dst * x.out_token +
                       (second ? h - a.t[0].heads : h) * x.out_head + off0;
                if (rotates) {
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        T &ra = LAYOUT == 0 ? f[u][0].e[2 * i % V] : f[u][0].e[i];
                        T &rb = LAYOUT == 0 ? f[u][0].e[(2 * i + 1) % V] : f[u][kFrags - 1].e[i];
                        const float va = to_f32(ra), vb = to_f32(rb);
                        // the last rotated chunk may hold plain features too
                        if (first + i < R) {
                            from_f32(ra, va * cs[i] - vb * sn[i]);
                            from_f32(rb, vb * cs[i] + va * sn[i]);
                        }
                    }
                }
                store_frag<T, V>(p, f[u][0]);
                if (LAYOUT == 1 && rotates) store_frag<T, V>(p + R, f[u][kFrags - 1]);
            }
        }
    }
}

template <typename T, int LAYOUT, int V>
static cudaError_t launch_rope(RopeArgs &a, cudaStream_t stream) {
    const int chunks = LAYOUT == 0 ? a.D / V : a.pairs / V + (a.D - 2 * a.pairs) / V;
    const int rows = 256 / chunks;
    const int64_t token_blocks = (a.N + rows - 1) / rows;
    const int heads = a.t[0].heads + (a.count > 1 ? a.t[1].heads : 0);
    // 16 heads a CTA (of 80 heads: 8 a CTA 582 us, 16 492, 40 506, 80 518: fewer
    // take the angles too often, more walk too far apart in memory); fewer where
    // that does not fill the GPU (four CTAs on each of the 148 SMs).
    int64_t splits = (4 * 148 + token_blocks * a.B - 1) / (token_blocks * a.B);
    if (splits < (heads + 15) / 16) splits = (heads + 15) / 16;
    if (splits > heads) splits = heads;
    a.heads_per_cta = static_cast<int>((heads + splits - 1) / splits);
    const int head_blocks = (heads + a.heads_per_cta - 1) / a.heads_per_cta;
    rope_kernel<T, LAYOUT, V><<<dim3(static_cast<unsigned>(token_blocks), head_blocks, a.B),
                                dim3(chunks, rows), 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace nabla

// wide: 16-byte accesses are possible on every view
cudaError_t nabla_launch_rope(nabla::RopeArgs &a, int dtype, int layout, int wide,
                              cudaStream_t stream) {
    using namespace nabla;
#define NABLA_ROPE(T, VW)                                                                     \
    return layout == 0 ? (wide ? launch_rope<T, 0, VW>(a, stream) : launch_rope<T, 0, 2>(a, stream)) \
                       : (wide ? launch_rope<T, 1, VW>(a, stream) : launch_rope<T, 1, 1>(a, stream));
    if (dtype == 0) NABLA_ROPE(__nv_bfloat16, 8)
    if (dtype == 1) NABLA_ROPE(__half, 8)
    NABLA_ROPE(float, 4)
#undef NABLA_ROPE
}
