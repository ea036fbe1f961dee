// Plan of the gated feed-forward block: see ffn_plan.h.
#include "ffn_plan.h"

#include <algorithm>

#include "tiles.h"

namespace mok {

namespace {

constexpr int64_t kUnits = 256;          // compute units of one MI355X
constexpr size_t kPartBytes = 64u << 20;   // most bytes of fp32 partials of one product
constexpr int kMaxSplits = 32;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

struct Carver {
    size_t off = 0;
    size_t take(size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes);
        return o;
    }
};

size_t part_bytes(int64_t T, int H, int I) {
    const int64_t widest = std::max<int64_t>(H, 2 * (int64_t)I);
    return (size_t)std::min<int64_t>((int64_t)kPartBytes, (int64_t)kMaxSplits * T * widest * 4);
}

// The tile height and split of a product of T rows, N columns (n_tiles tiles
// of them) and `steps` K-steps: the least estimated time over the choices,
// from the rounds of tiles over the compute units, the time of a K-step, and
// the traffic of the partials. Depends on the shape alone, so the bits of a
// result do too.
FfnSplit choose(int64_t T, int64_t N, int64_t n_tiles, int steps, bool mx) {
    FfnSplit best{256, 1, steps};
    double least = 1e30;
    for (int bm : {256, 128}) {
        const double step_us = bm == 256 ? (mx ? 0.9 : 0.85) : (mx ? 0.55 : 0.5);
        for (int s = 1; s <= kMaxSplits; ++s) {
            int len = (int)ceil_div(steps, s);
            if (mx) len = (len + 1) / 2 * 2;   // whole 128-value runs: one dword of scales a row
            const int eff = (int)ceil_div(steps, len);
            if (s > 1 && (eff != s || len < 4)) continue;
            if (s > 1 && (size_t)(eff * T * N * 4) > kPartBytes) continue;
            const int64_t rounds = ceil_div(ceil_div(T, bm) * n_tiles * eff, kUnits);
            double us = (double)rounds * (len * step_us + 6.0);
            if (s > 1) us += 5.0 + (double)eff * T * N * 8 / 4.0e6;
            if (us < least) {
                least = us;
                best = FfnSplit{bm, eff, len};
            }
        }
    }
    return best;
}

}  // namespace

mok_status make_ffn_plan(int64_t T, int32_t H, int32_t I, int32_t precision, FfnPlan *out) {
    if (T < 0 || H <= 0 || I <= 0) return MOK_ERROR_INVALID_VALUE;
    if (precision != MOK_BF16 && precision != MOK_MXFP8) return MOK_ERROR_INVALID_VALUE;
    const bool mx = precision == MOK_MXFP8;
    const int q = mx ? 128 : 64;
    if (H % q || I % q) return MOK_ERROR_INVALID_VALUE;
    // the layer's own bounds: 32-bit byte offsets into x / out, h / dh and a weight gradient
    if (T >= (int64_t(1) << 31)) return MOK_ERROR_INVALID_VALUE;
    if (T * (int64_t)H * 2 >= (int64_t(1) << 31)) return MOK_ERROR_INVALID_VALUE;
    if (T * (int64_t)I * 4 >= (int64_t(1) << 31)) return MOK_ERROR_INVALID_VALUE;
    if (((int64_t)H + 256) * I * 2 >= (int64_t(1) << 31) || ((int64_t)I + 256) * H * 2 >= (int64_t(1) << 31))
        return MOK_ERROR_INVALID_VALUE;
    FfnPlan p{};
    p.T = T;
    p.H = H;
    p.I = I;
    p.mx = mx;
    const int k = mx ? 64 : 32;
    p.gate_up = choose(T, 2 * (int64_t)I, ceil_div(I, kTileN / 2), H / k, mx);
    p.down = choose(T, H, ceil_div(H, kTileN), I / k, mx);
    p.da = choose(T, I, ceil_div(I, kTileN), H / k, mx);
    p.dx = choose(T, H, ceil_div(H, kTileN), 2 * I / k, mx);
    const int64_t big = ceil_div(2 * (int64_t)I, 256) * ceil_div(H, 256) + ceil_div(H, 256) * ceil_div(I, 256);
    p.wgrad_bm = big < kUnits ? 128 : 256;
    Carver w;
    p.part = w.take(part_bytes(T, H, I));
    p.a = w.take((size_t)T * I * 2);
    p.dh = w.take((size_t)T * I * 4);
    if (mx) {
        p.a_q = w.take((size_t)T * I);
        p.a_qs = w.take((size_t)T * I / 32);
        p.dh_q = w.take((size_t)T * I * 2);
        p.dh_qs = w.take((size_t)T * I / 16);
        p.dy_q = w.take((size_t)T * H);
        p.dy_qs = w.take((size_t)T * H / 32);
    }
    p.total = std::max<size_t>(w.off, 256);
    *out = p;
    return MOK_OK;
}

}  // namespace mok
