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

// Workgroups of a product of n tiles (ffn_grid, wgrad_grid).
int64_t grid(int64_t n) { return ceil_div(n, kGridStep) * kGridStep; }

size_t part_bytes(int64_t T, int H, int I) {
    const int64_t widest = std::max<int64_t>(H, 2 * (int64_t)I);
    return (size_t)std::min<int64_t>((int64_t)kPartBytes, (int64_t)kMaxSplits * T * widest * 4);
}

// The tile height and split of a product of T rows, N columns (n_tiles tiles
// of them) and `steps` K-steps: the least estimated time over the choices,
// from the rounds of tiles over the compute units, the time of a K-step, and
// the join with its partials' traffic. The constants were fitted to kernel
// traces of 15 lengths from 3 to 4,096 rows at 7,168 x 2,048, 4,096 x 1,024,
// 2,048 x 768, 1,024 x 512 and 512 x 2,048: the choices are 1.5% slower than the
// best measured ones in the mean, 25% at most.
// Depends on the shape alone, so the bits of a result do too.
FfnSplit choose(int64_t T, int64_t N, int64_t n_tiles, int steps, bool mx) {
    FfnSplit best{256, 1, steps};
    double least = 1e30;
    for (int bm : {256, 128}) {
        const double step_us = bm == 256 ? (mx ? 0.8 : 0.75) : (mx ? 0.53 : 0.5);
        const int64_t tiles = ceil_div(T, bm) * n_tiles;
        for (int s = 1; s <= kMaxSplits; ++s) {
            int len = (int)ceil_div(steps, s);
            if (mx) len = (len + 1) / 2 * 2;   // whole 128-value runs: one dword of scales a row
            if (s > 1 && len < 2) break;
            if (s > 1 && ceil_div(steps, len) != s) continue;
            if (s > 1 && (size_t)(s * T * N * 4) > kPartBytes) break;
            double us = (double)ceil_div(tiles * s, kUnits) * (len * step_us + 5.0);
            if (s > 1) us += 6.0 + 0.1 * s + (double)s * T * N * 8 / 5.0e6;
            if (us < least) {
                least = us;
                best = FfnSplit{bm, s, len};
            }
        }
    }
    return best;
}

// The few-rows forward, where it is faster than the tiles (GPU time of a call):
// one row always (7,168 x 2,048 BF16 24 us against 28, MXFP8 16 against 24;
// 1,024 x 512 12 against 16 and 7 against 15); two rows in MXFP8 (21 against 24,
// 10 against 15) and in BF16 up to 2^23 weights a matrix (4,096 x 1,024 19 us
// against 24; 7,168 x 2,048 32 against 29). Its buffers in LDS stay under
// 64 KiB (the rows of a in fp32, in MXFP8 with a scale for each 32 values), and
// BF16 cuts the gate/up product into at most 16 runs of at most 2,048 rows,
// about one workgroup per compute unit.
void plan_few(FfnPlan &p) {
    p.few_runs = p.few_run_rows = 0;
    if (p.T < 1 || p.T > kFewRows || p.T * p.I > 15 * 1024 || p.H > 16 * 2048) return;
    if (p.T > 1 && !p.mx && (int64_t)p.H * p.I > (int64_t(1) << 23)) return;
    p.few_runs = 1;
    if (p.mx) return;
    const int64_t strips = p.I / 64, groups = p.H / 64;
    int64_t runs = std::min<int64_t>(std::max<int64_t>(kUnits / strips, 1), 16);
    runs = std::max(runs, ceil_div(groups, 2048 / 64));
    const int64_t len = ceil_div(groups, runs);
    p.few_run_rows = (int)len * 64;
    p.few_runs = (int)ceil_div(groups, len);
}

}  // namespace

mok_status make_ffn_plan(int64_t T, int32_t H, int32_t I, int32_t precision, FfnPlan *out) {
    if (T < 0 || H <= 0 || I <= 0) return MOK_ERROR_INVALID_VALUE;
    if (precision != MOK_BF16 && precision != MOK_MXFP8) return MOK_ERROR_INVALID_VALUE;
    const bool mx = precision == MOK_MXFP8;
    const int q = mx ? 128 : 64;
    if (H % q || I % q) return MOK_ERROR_INVALID_VALUE;
    // 256 rows of a tile at 8 I or 4 H bytes each (fp32 partials) stay below 2^32, so that the offset of a row
    // past the tile's valid ones never wraps into them
    if (H > (1 << 20) || I > (1 << 20)) return MOK_ERROR_INVALID_VALUE;
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
    plan_few(p);
    const int k = mx ? 64 : 32;
    p.gate_up = choose(T, 2 * (int64_t)I, ceil_div(I, kTileN / 2), H / k, mx);
    p.down = choose(T, H, ceil_div(H, kTileN), I / k, mx);
    p.da = choose(T, I, ceil_div(I, kTileN), H / k, mx);
    p.dx = choose(T, H, ceil_div(H, kTileN), 2 * I / k, mx);
    const int64_t big = ceil_div(2 * (int64_t)I, 256) * ceil_div(H, 256) + ceil_div(H, 256) * ceil_div(I, 256);
    p.wgrad_bm = big < kUnits ? 128 : 256;
    // dx and the weight gradients in one launch, on 128 rows both: with more tiles
    // than compute units, two workgroups a unit (1,001 and 2,048 rows of
    // 4,096 x 1,024: backward 84 -> 78 and 142 -> 131 us); with fewer, the deeper
    // ring (2,048 rows of 1,024 x 512: 60 us against 71)
    p.grads_two = !mx && p.dx.bm == 128 && p.wgrad_bm == 128 &&
                  grid(ceil_div(H, 128) * ceil_div(2 * (int64_t)I, kTileN)) +
                          grid(ceil_div(I, 128) * ceil_div(H, kTileN)) +
                          grid(ceil_div(T, 128) * ceil_div(H, kTileN) * p.dx.splits) >
                      kUnits;
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
