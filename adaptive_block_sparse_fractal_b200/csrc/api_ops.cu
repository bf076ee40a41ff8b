// C ABI of the calls around the grid attention (declared in include/nabla.h):
// rotary positions, packed-sequence attention, the paged key-value cache.
// Argument checks, workspace layout, kernel dispatch; every host-detectable
// error is returned before anything is enqueued.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/nabla.h"
#include "packed.cuh"
#include "paged.cuh"
#include "rope.cuh"
#include "views.h"

// launchers (rope.cu, packed_fwd.cu, packed_bwd.cu, paged.cu)
cudaError_t nabla_launch_rope(nabla::RopeArgs &a, int dtype, int layout, int wide,
                              cudaStream_t stream);
cudaError_t nabla_launch_packed_fwd(const nabla::packed::Args &a, int D, cudaStream_t stream);
cudaError_t nabla_launch_packed_bwd(const nabla::packed::Args &a, int D, int64_t q_tiles,
                                    int64_t key_tiles, cudaStream_t stream);
cudaError_t nabla_launch_append(const nabla::AppendArgs &a, cudaStream_t stream);
cudaError_t nabla_launch_paged(const nabla::PagedArgs &a, cudaStream_t stream);

namespace {

constexpr size_t kStatusBytes = 256;

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? NABLA_OK : NABLA_ERR_CUDA; }
cudaStream_t as_stream(nabla_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// (the kernels take scale * log2(e))
bool scale_ok(float s) { return s > 0.f && std::isfinite(s * 1.4426950408889634f); }

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (ws == nullptr || bytes < need) return NABLA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return NABLA_ERR_ALIGN;
    return NABLA_OK;
}

using nabla::views::Box;
using nabla::views::disjoint;
using nabla::views::flat;
using nabla::views::make_box;
using nabla::views::multiple_of_16;
using nabla::views::same_view;
using nabla::views::self_disjoint;

// Whether no output shares a byte with an input or with another output.
bool apart(std::initializer_list<const Box *> outs, std::initializer_list<const Box *> ins) {
    for (const Box *const *o = outs.begin(); o != outs.end(); ++o) {
        for (const Box *i : ins)
            if (!disjoint(**o, *i)) return false;
        for (const Box *const *p = outs.begin(); p != o; ++p)
            if (!disjoint(**o, **p)) return false;
    }
    return true;
}

Box ints(const int32_t *p, int64_t n) { return flat(p, 4 * n); }

// ---------------------------------------------------------------------------
// packed attention
// ---------------------------------------------------------------------------
constexpr int64_t kMaxPackedRows = (1ll << 31) - 1024;

bool packed_shape_ok(const nabla_packed *s) {
    return s->seqs >= 1 && s->heads >= 1 && s->heads <= 65535 && s->heads_kv >= 1 &&
           s->heads % s->heads_kv == 0 &&
           s->heads / s->heads_kv <= 128 && (s->D == 64 || s->D == 128) && s->total_q >= 0 && s->total_k >= 0 &&
           s->total_k <= kMaxPackedRows && s->total_q <= kMaxPackedRows / s->heads &&
           s->seqs <= (1 << 24);
}

// Tokens of a row tile of the forward: 128 rows hold them for all heads of a group.
int tile_tokens(const nabla_packed *s) { return 128 / (s->heads / s->heads_kv); }

// Forward units (two row tiles) of all key heads, at most: every sequence may end inside one.
int64_t fwd_units(const nabla_packed *s) {
    return (s->total_q / (2 * tile_tokens(s)) + s->seqs) * s->heads_kv;
}

// Splits of the key range, where the units leave SMs idle: the number that
// makes a CTA's walk over its share of the keys (1.2 us per 128) and the join (5
// us, 0.3 a part, and the parts written and read at about 4 TB/s) shortest, taking the
// average sequence for all.  Measured, 1 split against the choice: 1 row on 4,096
// keys, 24/8 heads, D = 128: 47 against 21 us; 16 rows on 16,384, 40/8 heads: 163
// against 33; 300 rows on 1,200 keep 1 split: 29 us against 37 with two.
int fwd_splits(const nabla_packed *s) {
    const int64_t most = 148 / fwd_units(s);
    const double walk = 1.2 * static_cast<double>(s->total_k) / s->seqs / 128.0;
    const double part = 8.0 * static_cast<double>(s->total_q) * s->heads * (s->D + 2) / 4e6;
    int best = 1;
    double time = walk;
    for (int n = 2; n <= most && n <= 32; ++n) {
        const double t = walk / n + 5.0 + (0.3 + part) * n;
        if (t < time) {
            time = t;
            best = n;
        }
    }
    return best;
}

size_t packed_ws(const nabla_packed *s, int op) {
    const int splits = fwd_splits(s);
    size_t n = 0;
    if (splits > 1)
        n = round256(sizeof(float) * splits * s->total_q * s->heads * (s->D + 2));
    if (op == NABLA_PACKED_BWD) {
        const size_t pad = static_cast<size_t>((s->total_q / 64 + s->seqs) * 64);
        const size_t b = 2 * round256(sizeof(float) * pad * s->heads);
        if (b > n) n = b;
    }
    return kStatusBytes + n;
}

nabla::packed::View dev_view(const nabla_view *v) {
    return {static_cast<__nv_bfloat16 *>(v->data), v->token, v->head};
}

int packed_view(const nabla_view *v, int64_t tokens, int heads, int D, bool written, Box *b) {
    if (v == nullptr) return NABLA_ERR_NULL;
    if (tokens == 0) return make_box(v, 1, heads, 0, D, 2, b) ? NABLA_OK : NABLA_ERR_PARAM;  // (empty)
    if (v->data == nullptr) return NABLA_ERR_NULL;
    if (!make_box(v, 1, heads, tokens, D, 2, b)) return NABLA_ERR_PARAM;
    if (!multiple_of_16(*b)) return NABLA_ERR_ALIGN;
    // the tensor maps of k, v, q, dout want distances above 0
    for (int i = 1; i < 3; ++i)
        if (b->n[i] > 1 && (b->stride[i] < 1 || b->stride[i] * 2 >= (1ll << 40)))
            return NABLA_ERR_PARAM;
    if (written && !self_disjoint(*b)) return NABLA_ERR_PARAM;
    return NABLA_OK;
}

int check_packed(const nabla_packed *s, const int32_t *cu_q, const int32_t *cu_k, int op, void *ws,
                 size_t bytes) {
    if (s == nullptr) return NABLA_ERR_NULL;
    if (!packed_shape_ok(s)) return NABLA_ERR_SHAPE;
    if (!scale_ok(s->scale) ||
        (s->causal & ~static_cast<int>(1u | NABLA_DEBUG_TIMEOUT)) != 0)
        return NABLA_ERR_PARAM;
    if (cu_q == nullptr || cu_k == nullptr) return NABLA_ERR_NULL;
    if (!aligned4(cu_q) || !aligned4(cu_k)) return NABLA_ERR_ALIGN;
    return check_workspace(ws, bytes, packed_ws(s, op));
}

nabla::packed::Args packed_args(const nabla_packed *s, const int32_t *cu_q, const int32_t *cu_k,
                                void *ws) {
    nabla::packed::Args a = {};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.status = static_cast<int *>(ws);
    a.total_q = s->total_q;
    a.total_k = s->total_k;
    a.seqs = s->seqs;
    a.heads = s->heads;
    a.heads_kv = s->heads_kv;
    a.group = s->heads / s->heads_kv;
    a.causal = s->causal & 1;
    a.tile_tokens = tile_tokens(s);
    a.splits = 1;
    a.c = s->scale * 1.4426950408889634f;
    a.scale = s->scale;
    a.stall = (s->causal & NABLA_DEBUG_TIMEOUT) != 0;
    a.limit = a.stall ? 1000000u : 1000000000u;  // 1 s per wait (1 ms when it is to expire)
    return a;
}

// ---------------------------------------------------------------------------
// paged cache
// ---------------------------------------------------------------------------
bool cache_shape_ok(const nabla_cache *c) {
    return c->pages >= 1 && c->page_size >= 1 && c->heads_kv >= 1 && c->D >= 8 && c->D % 8 == 0 &&
           c->D <= 256 && c->seqs >= 0 && c->table_width >= 1 && c->heads_kv <= (1 << 20);
}

int check_cache(const nabla_cache *c, bool written, Box bx[2], nabla::CacheArgs *a) {
    if (c->k.data == nullptr || c->v.data == nullptr || c->table == nullptr) return NABLA_ERR_NULL;
    if (!aligned4(c->table)) return NABLA_ERR_ALIGN;
    const nabla_view *v[2] = {&c->k, &c->v};
    for (int i = 0; i < 2; ++i) {
        if (!make_box(v[i], c->pages, c->heads_kv, c->page_size, c->D, 2, &bx[i]))
            return NABLA_ERR_PARAM;
        if (!multiple_of_16(bx[i])) return NABLA_ERR_ALIGN;
        if (written && !self_disjoint(bx[i])) return NABLA_ERR_PARAM;
    }
    a->k = static_cast<__nv_bfloat16 *>(c->k.data);
    a->v = static_cast<__nv_bfloat16 *>(c->v.data);
    a->k_page = bx[0].stride[0];
    a->k_head = bx[0].stride[1];
    a->k_token = bx[0].stride[2];
    a->v_page = bx[1].stride[0];
    a->v_head = bx[1].stride[1];
    a->v_token = bx[1].stride[2];
    a->table = c->table;
    a->pages = c->pages;
    a->page_size = c->page_size;
    a->heads_kv = c->heads_kv;
    a->D = c->D;
    a->seqs = c->seqs;
    a->width = c->table_width;
    return NABLA_OK;
}

size_t paged_ws(const nabla_cache *c) {
    return kStatusBytes + round256(sizeof(int) * nabla::kPagedCtas) +
           sizeof(float) * 2 * nabla::kPagedCtas * nabla::kPagedHeads * (c->D + 2);
}

}  // namespace

extern "C" {

int nabla_rope(const nabla_rope_params *p, int B, int T, int H, int W, int P, int count,
               const int *heads, const nabla_view *in, const nabla_view *out, const int32_t *pos,
               int64_t pos_batch, int pos_axes, nabla_stream_t stream) {
    if (p == nullptr || heads == nullptr || in == nullptr || out == nullptr) return NABLA_ERR_NULL;
    if (B < 0 || T < 0 || H < 0 || W < 0 || count < 1 || count > 2) return NABLA_ERR_SHAPE;
    if (p->dtype < NABLA_BF16 || p->dtype > NABLA_FP32 ||
        (p->layout != NABLA_ROPE_ADJACENT && p->layout != NABLA_ROPE_HALVES) ||
        (p->flags & ~(NABLA_ROPE_INVERSE | NABLA_ROPE_FLAT_IN | NABLA_ROPE_FLAT_OUT)) != 0)
        return NABLA_ERR_PARAM;
    if (p->D < 2 || p->D > 2 * nabla::kRopeMaxPairs || p->D % 2 != 0) return NABLA_ERR_SHAPE;
    int R = 0;
    for (int a = 0; a < 3; ++a) {
        if (p->pairs[a] < 0 || p->pairs[a] > nabla::kRopeMaxPairs) return NABLA_ERR_PARAM;
        R += p->pairs[a];
        if (p->pairs[a] > 0 && (!(p->theta[a] > 0.0) || !std::isfinite(p->theta[a]) ||
                                !std::isfinite(p->scale[a]) || !std::isfinite(p->offset[a])))
            return NABLA_ERR_PARAM;
        if (p->pairs[a] > 0 && pos != nullptr && a >= pos_axes) return NABLA_ERR_PARAM;
    }
    if (R < 1 || 2 * R > p->D) return NABLA_ERR_PARAM;
    const bool flat = (p->flags & (NABLA_ROPE_FLAT_IN | NABLA_ROPE_FLAT_OUT)) != 0;
    if (flat && (P < 1 || H % P != 0 || W % P != 0)) return NABLA_ERR_SHAPE;
    if (pos != nullptr && (pos_axes < 1 || pos_axes > 3 || pos_batch < 0)) return NABLA_ERR_PARAM;
    if (!aligned4(pos)) return NABLA_ERR_ALIGN;
    for (int i = 0; i < count; ++i)
        if (heads[i] < 0 || heads[i] > 32767) return NABLA_ERR_SHAPE;
    if (B == 0 || T == 0 || H == 0 || W == 0) return NABLA_OK;  // empty
    const int64_t N = static_cast<int64_t>(T) * H <= INT32_MAX / W ? static_cast<int64_t>(T) * H * W : -1;
    if (N < 0 || N > INT32_MAX - 256 || B > 65535) return NABLA_ERR_SHAPE;
    const int size = p->dtype == NABLA_FP32 ? 4 : 2;
    const int vec = 16 / size;
    bool wide = p->D % vec == 0 && (p->layout == NABLA_ROPE_ADJACENT || R % vec == 0);
    Box bi[2], bo[2];
    int n = 0;
    nabla::RopeArgs a = {};
    for (int i = 0; i < count; ++i) {
        if (heads[i] == 0) continue;  // nothing of this tensor
        if (in[i].data == nullptr || out[i].data == nullptr) return NABLA_ERR_NULL;
        if (!make_box(&in[i], B, heads[i], N, p->D, size, &bi[n]) ||
            !make_box(&out[i], B, heads[i], N, p->D, size, &bo[n]))
            return NABLA_ERR_PARAM;
        if (bi[n].lo % size != 0 || bo[n].lo % size != 0) return NABLA_ERR_ALIGN;
        wide = wide && multiple_of_16(bi[n]) && multiple_of_16(bo[n]);
        if (!self_disjoint(bo[n])) return NABLA_ERR_PARAM;
        a.t[n].in = in[i].data;
        a.t[n].out = out[i].data;
        a.t[n].in_batch = bi[n].stride[0];
        a.t[n].in_head = bi[n].stride[1];
        a.t[n].in_token = bi[n].stride[2];
        a.t[n].out_batch = bo[n].stride[0];
        a.t[n].out_head = bo[n].stride[1];
        a.t[n].out_token = bo[n].stride[2];
        a.t[n].heads = heads[i];
        ++n;
    }
    if (n == 0) return NABLA_OK;
    // in place: each thread writes exactly the elements it has read, if both
    // sides have the same order (both flattened counts as the same)
    const bool same_order = ((p->flags & NABLA_ROPE_FLAT_IN) != 0) == ((p->flags & NABLA_ROPE_FLAT_OUT) != 0);
    const Box places = ints(pos, (pos_batch > 0 ? (B - 1) * pos_batch : 0) + N * pos_axes);
    for (int i = 0; i < n; ++i)
        if (!disjoint(bo[i], places)) return NABLA_ERR_PARAM;
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (!(i == j && same_order && same_view(bo[i], bi[i])) && !disjoint(bo[i], bi[j]))
                return NABLA_ERR_PARAM;
            if (i < j && !disjoint(bo[i], bo[j])) return NABLA_ERR_PARAM;
        }
    a.count = n;
    a.B = B;
    a.N = static_cast<int>(N);
    a.T = T;
    a.H = H;
    a.W = W;
    a.P = flat ? P : 1;
    a.D = p->D;
    a.pairs = R;
    a.flat_in = (p->flags & NABLA_ROPE_FLAT_IN) != 0;
    a.flat_out = (p->flags & NABLA_ROPE_FLAT_OUT) != 0;
    a.pos = pos;
    a.pos_batch = pos_batch;
    a.pos_axes = pos_axes;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    // largest distance from 0 of a position on each axis
    const double reach[3] = {pos != nullptr ? 2147483648.0 : T, pos != nullptr ? 2147483648.0 : H,
                             pos != nullptr ? 2147483648.0 : W};
    for (int ax = 0, at = 0; ax < 3; ++ax) {
        a.offset[ax] = p->pairs[ax] > 0 ? p->offset[ax] : 0.0;
        // theta^(-i / n): a power for every eighth pair, products of up to 7 ratios
        // between them (1e-15 relative; a pow a pair took 3 us of the call)
        const double ratio = p->pairs[ax] > 0 ? std::pow(p->theta[ax], -1.0 / p->pairs[ax]) : 0.0;
        double f = 1.0;
        for (int i = 0; i < p->pairs[ax]; ++i, ++at) {
            f = i % 8 == 0 ? std::pow(p->theta[ax], -static_cast<double>(i) / p->pairs[ax]) : f * ratio;
            a.axis[at] = static_cast<int8_t>(ax);
            a.turn[at] = ((p->flags & NABLA_ROPE_INVERSE) ? -1.0 : 1.0) * p->scale[ax] * f / kTwoPi;
            // the reduction to an eighth of a turn holds below 2^49 turns (float64 knows no
            // more of the angle there); this refuses infinities and NaN as well
            if (!((reach[ax] + std::fabs(a.offset[ax])) * std::fabs(a.turn[at]) < 0x1p49)) return NABLA_ERR_PARAM;
        }
    }
    return cuda_status(nabla_launch_rope(a, p->dtype, p->layout, wide, as_stream(stream)));
}

size_t nabla_packed_workspace_size(const nabla_packed *shape, int op) {
    if (shape == nullptr || !packed_shape_ok(shape) ||
        (op != NABLA_PACKED_FWD && op != NABLA_PACKED_BWD))
        return 0;
    return packed_ws(shape, op);
}

int nabla_attn_packed_fwd(const nabla_packed *shape, const nabla_view *q, const nabla_view *k,
                          const nabla_view *v, const int32_t *cu_q, const int32_t *cu_k,
                          const nabla_view *o, float *lse, void *workspace, size_t workspace_bytes,
                          nabla_stream_t stream) {
    int st = check_packed(shape, cu_q, cu_k, NABLA_PACKED_FWD, workspace, workspace_bytes);
    if (st != NABLA_OK) return st;
    Box bq, bk, bv, bo;
    if ((st = packed_view(q, shape->total_q, shape->heads, shape->D, false, &bq)) != NABLA_OK ||
        (st = packed_view(k, shape->total_k, shape->heads_kv, shape->D, false, &bk)) != NABLA_OK ||
        (st = packed_view(v, shape->total_k, shape->heads_kv, shape->D, false, &bv)) != NABLA_OK ||
        (st = packed_view(o, shape->total_q, shape->heads, shape->D, true, &bo)) != NABLA_OK)
        return st;
    if (!aligned4(lse)) return NABLA_ERR_ALIGN;
    const Box bl = flat(lse, 4 * shape->total_q * shape->heads), bw = flat(workspace, packed_ws(shape, NABLA_PACKED_FWD)),
              cq = ints(cu_q, shape->seqs + 1), ck = ints(cu_k, shape->seqs + 1);
    if (!apart({&bo, &bl, &bw}, {&bq, &bk, &bv, &cq, &ck})) return NABLA_ERR_PARAM;
    const int64_t units = fwd_units(shape);
    const int splits = fwd_splits(shape);
    if (units > INT32_MAX / splits) return NABLA_ERR_SHAPE;
    cudaStream_t s = as_stream(stream);
    // the status word and the unit counter behind it; with no more units than
    // CTAs the counter is not used, and the kernel writes the status itself
    if (shape->total_q == 0 || units * splits > nabla::packed::kSms)
        if (cudaMemsetAsync(workspace, 0, 2 * sizeof(int), s) != cudaSuccess) return NABLA_ERR_CUDA;
    if (shape->total_q == 0) return NABLA_OK;
    nabla::packed::Args a = packed_args(shape, cu_q, cu_k, workspace);
    a.q = dev_view(q);
    a.k = dev_view(k);
    a.v = dev_view(v);
    a.o = dev_view(o);
    a.lse = lse;
    a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kStatusBytes);
    a.splits = splits;
    a.units = static_cast<uint32_t>(units * splits);
    return cuda_status(nabla_launch_packed_fwd(a, shape->D, s));
}

int nabla_attn_packed_bwd(const nabla_packed *shape, const nabla_view *q, const nabla_view *k,
                          const nabla_view *v, const nabla_view *o, const nabla_view *dout,
                          const float *lse, const int32_t *cu_q, const int32_t *cu_k,
                          const nabla_view *dq, const nabla_view *dk, const nabla_view *dv,
                          void *workspace, size_t workspace_bytes, nabla_stream_t stream) {
    int st = check_packed(shape, cu_q, cu_k, NABLA_PACKED_BWD, workspace, workspace_bytes);
    if (st != NABLA_OK) return st;
    const nabla_view *in[5] = {q, k, v, o, dout}, *out[3] = {dq, dk, dv};
    Box bi[5], bo[3];
    const bool of_q[5] = {true, false, false, true, true}, out_q[3] = {true, false, false};
    auto view = [&](const nabla_view *x, bool is_q, bool written, Box *b) {
        return packed_view(x, is_q ? shape->total_q : shape->total_k, is_q ? shape->heads : shape->heads_kv,
                           shape->D, written, b);
    };
    for (int i = 0; i < 5; ++i)
        if ((st = view(in[i], of_q[i], false, &bi[i])) != NABLA_OK) return st;
    for (int i = 0; i < 3; ++i)
        if ((st = view(out[i], out_q[i], true, &bo[i])) != NABLA_OK) return st;
    if (shape->total_q > 0 && lse == nullptr) return NABLA_ERR_NULL;
    if (!aligned4(lse)) return NABLA_ERR_ALIGN;
    // the three kernels read the inputs while the first outputs are written
    const Box bl = flat(lse, 4 * shape->total_q * shape->heads), bw = flat(workspace, packed_ws(shape, NABLA_PACKED_BWD)),
              cq = ints(cu_q, shape->seqs + 1), ck = ints(cu_k, shape->seqs + 1);
    if (!apart({&bo[0], &bo[1], &bo[2], &bw}, {&bi[0], &bi[1], &bi[2], &bi[3], &bi[4], &bl, &cq, &ck}))
        return NABLA_ERR_PARAM;
    const int64_t G = shape->heads / shape->heads_kv;
    const int64_t q_tiles = shape->total_q / 64 + shape->seqs;
    const int64_t row_tiles = shape->total_q * G / 128 + shape->seqs;
    const int64_t key_tiles = shape->total_k / 128 + shape->seqs;
    if (row_tiles * shape->heads_kv > INT32_MAX || key_tiles * shape->heads_kv > INT32_MAX)
        return NABLA_ERR_SHAPE;
    cudaStream_t s = as_stream(stream);
    // the status word, the unit counter and the verdict on the borders behind it
    if (cudaMemsetAsync(workspace, 0, 3 * sizeof(int), s) != cudaSuccess) return NABLA_ERR_CUDA;
    if (shape->total_q == 0 && shape->total_k == 0) return NABLA_OK;
    nabla::packed::Args a = packed_args(shape, cu_q, cu_k, workspace);
    a.q = dev_view(q);
    a.k = dev_view(k);
    a.v = dev_view(v);
    a.o = dev_view(o);
    a.dout = dev_view(dout);
    a.dq = dev_view(dq);
    a.dk = dev_view(dk);
    a.dv = dev_view(dv);
    a.lse = const_cast<float *>(lse);
    a.pad_rows = q_tiles * 64;
    a.units = static_cast<uint32_t>(row_tiles * shape->heads_kv);
    unsigned char *w = static_cast<unsigned char *>(workspace) + kStatusBytes;
    a.pad_l = reinterpret_cast<float *>(w);
    a.pad_d = reinterpret_cast<float *>(w + round256(sizeof(float) * a.pad_rows * shape->heads));
    return cuda_status(nabla_launch_packed_bwd(a, shape->D, q_tiles, key_tiles, s));
}

int nabla_cache_append(const nabla_cache *cache, const nabla_view *k, const nabla_view *v,
                       int64_t total, const int32_t *starts, const int32_t *cu, void *workspace,
                       size_t workspace_bytes, nabla_stream_t stream) {
    if (cache == nullptr || k == nullptr || v == nullptr) return NABLA_ERR_NULL;
    if (!cache_shape_ok(cache) || total < 0 || total > INT32_MAX) return NABLA_ERR_SHAPE;
    if (cu == nullptr && total != cache->seqs) return NABLA_ERR_SHAPE;  // one row a sequence
    nabla::AppendArgs a = {};
    if (workspace != nullptr) {
        const int st = check_workspace(workspace, workspace_bytes, kStatusBytes);
        if (st != NABLA_OK) return st;
        a.status = static_cast<int *>(workspace);
    }
    Box pool[2], bk, bv;
    const bool work = total > 0 && cache->seqs > 0;
    if (work) {
        const int st = check_cache(cache, true, pool, &a.c);
        if (st != NABLA_OK) return st;
        if (k->data == nullptr || v->data == nullptr || starts == nullptr) return NABLA_ERR_NULL;
        if (!aligned4(starts) || !aligned4(cu)) return NABLA_ERR_ALIGN;
        if (!make_box(k, 1, cache->heads_kv, total, cache->D, 2, &bk) ||
            !make_box(v, 1, cache->heads_kv, total, cache->D, 2, &bv))
            return NABLA_ERR_PARAM;
        if (!multiple_of_16(bk) || !multiple_of_16(bv)) return NABLA_ERR_ALIGN;
        // K and V may be slices of one buffer, but share no row; rows that lie in a pool
        // could be overwritten before they are read
        const Box bw = flat(workspace, kStatusBytes), bs = ints(starts, cache->seqs), bc = ints(cu, cache->seqs + 1ll),
                  bt = ints(cache->table, static_cast<int64_t>(cache->seqs) * cache->table_width);
        if (!apart({&pool[0], &pool[1], &bw}, {&bk, &bv, &bs, &bc, &bt})) return NABLA_ERR_PARAM;
    }
    cudaStream_t s = as_stream(stream);
    // a few rows: one CTA of the launch looks at all of them and writes the status
    // itself, which saves the memset (1.5 us of an 11 us call)
    a.status_by_kernel = work && total <= 256;
    if (workspace != nullptr && !a.status_by_kernel &&
        cudaMemsetAsync(workspace, 0, sizeof(int), s) != cudaSuccess)
        return NABLA_ERR_CUDA;
    if (!work) return NABLA_OK;
    a.k = static_cast<const __nv_bfloat16 *>(k->data);
    a.v = static_cast<const __nv_bfloat16 *>(v->data);
    a.k_head = bk.stride[1];
    a.k_token = bk.stride[2];
    a.v_head = bv.stride[1];
    a.v_token = bv.stride[2];
    a.starts = starts;
    a.cu = cu;
    a.total = total;
    return cuda_status(nabla_launch_append(a, s));
}

size_t nabla_paged_workspace_size(const nabla_cache *cache, int heads) {
    if (cache == nullptr || !cache_shape_ok(cache) || (cache->D != 64 && cache->D != 128) ||
        heads < 1 || heads % cache->heads_kv != 0)
        return 0;
    return paged_ws(cache);
}

int nabla_attn_paged(const nabla_cache *cache, int heads, float scale, const nabla_view *q,
                     const int32_t *lens, const nabla_view *o, float *lse, void *workspace,
                     size_t workspace_bytes, nabla_stream_t stream) {
    if (cache == nullptr || q == nullptr || o == nullptr) return NABLA_ERR_NULL;
    if (nabla_paged_workspace_size(cache, heads) == 0) return NABLA_ERR_SHAPE;
    if (static_cast<int64_t>(cache->seqs) * heads > INT32_MAX) return NABLA_ERR_SHAPE;
    if (!scale_ok(scale)) return NABLA_ERR_PARAM;
    int st = check_workspace(workspace, workspace_bytes, paged_ws(cache));
    if (st != NABLA_OK) return st;
    cudaStream_t s = as_stream(stream);
    if (cache->seqs == 0)
        return cuda_status(cudaMemsetAsync(workspace, 0, sizeof(int), s));
    nabla::PagedArgs a = {};
    Box pool[2], bq, bo;
    if ((st = check_cache(cache, false, pool, &a.c)) != NABLA_OK) return st;
    if (q->data == nullptr || o->data == nullptr || lens == nullptr) return NABLA_ERR_NULL;
    if (!aligned4(lens) || !aligned4(lse)) return NABLA_ERR_ALIGN;
    if (!make_box(q, 1, heads, cache->seqs, cache->D, 2, &bq) ||
        !make_box(o, 1, heads, cache->seqs, cache->D, 2, &bo))
        return NABLA_ERR_PARAM;
    if (!multiple_of_16(bq) || !multiple_of_16(bo)) return NABLA_ERR_ALIGN;
    const Box bl = flat(lse, 4ll * cache->seqs * heads), bw = flat(workspace, paged_ws(cache)), bn = ints(lens, cache->seqs),
              bt = ints(cache->table, static_cast<int64_t>(cache->seqs) * cache->table_width);
    if (!self_disjoint(bo) || !apart({&bo, &bl, &bw}, {&bq, &pool[0], &pool[1], &bn, &bt})) return NABLA_ERR_PARAM;
    a.q = static_cast<const __nv_bfloat16 *>(q->data);
    a.o = static_cast<__nv_bfloat16 *>(o->data);
    a.q_head = bq.stride[1];
    a.q_token = bq.stride[2];
    a.o_head = bo.stride[1];
    a.o_token = bo.stride[2];
    a.lens = lens;
    a.lse = lse;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    a.status = reinterpret_cast<int *>(w);
    a.flags = reinterpret_cast<int *>(w + kStatusBytes);
    a.part = reinterpret_cast<float *>(w + kStatusBytes + round256(sizeof(int) * nabla::kPagedCtas));
    a.c2 = scale * 1.4426950408889634f;
    a.heads = heads;
    a.group = heads / cache->heads_kv;
    a.chunks = (a.group + nabla::kPagedHeads - 1) / nabla::kPagedHeads;
    a.ctas = nabla::kPagedCtas;
    return cuda_status(nabla_launch_paged(a, s));
}

}  // extern "C"
