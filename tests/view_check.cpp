// C entries of csrc/views.h for its test.
#include "../adaptive_block_sparse_fractal_b200/csrc/views.h"

using namespace nabla::views;

// box: address, extents and distances of [batch, head, token], D, element size
static bool box(const int64_t *x, Box *b) {
    const nabla_view v = {reinterpret_cast<void *>(x[0]), x[4], x[5], x[6]};
    return make_box(&v, x[1], x[2], x[3], x[7], static_cast<int>(x[8]), b);
}
// 1, 0, or -1 for a view that is refused
extern "C" int view_disjoint(const int64_t *x, const int64_t *y) {
    Box a, b;
    return !box(x, &a) || !box(y, &b) ? -1 : disjoint(a, b);
}
extern "C" int view_self_disjoint(const int64_t *x) {
    Box a;
    return !box(x, &a) ? -1 : self_disjoint(a);
}
