// Plan of the products on blocks of 128: see fp8_plan.h.
//
// Each choice is the least estimated time in us, from the rounds of tiles over the
// compute units, the time of a K-block, the weights' bytes, and the join of runs with
// its partials' traffic. The constants were fitted to some 40 shapes timed in a graph
// of calls, 1 to 16,384 rows by 1,024 to 14,336 columns, one product and 4 to 16
// experts. Some of them, us (the choice marked *):
//   rows x N x K              few rows at 16 / 32 / 64   128-row tiles in 1 / 4 / 8 runs   256-row tiles
//   1 x 4,096 x 7,168         7.7* / 8.7 / 11.2          44 / 19 / 14                      44
//   32 x 4,096 x 7,168        16.3 / 12.7* / 16.3        44 / 20 / 15.5                    45
//   64 x 7,168 x 2,048        19 / 11.9 / 10.1*          16.9 / 15.7 / 18.9                17.1
//   64 x 4,096 x 7,168        33 / 27 / 26               44 / 20.7 / 17.3*                 45
//   512 x 4,096 x 7,168       228 / 170 / 162            50 / 32* / 48                     51
//   2,048 x 7,168 x 2,048     495 / 387 / 311            41 / 122 / 242                    33*
//   16 of 16 experts, 7,168 x 2,048   42* / 40 / 61      47.8 / 75 / 108                   49
// It depends on the shape alone, so the bits of a result do too.
#include "fp8_plan.h"

#include <algorithm>

namespace mok {

namespace {

constexpr int64_t kUnits = 256;              // compute units of one MI355X
constexpr int kMostRuns = 32;
constexpr int64_t kPartBytes = 64 << 20;     // most bytes of partials
// Workgroups stay within one grid of fewer than 2^32 threads.
constexpr int64_t kMostGroups = (1 << 23) - 512;
constexpr double kTraffic = 5.0e6;           // bytes per us: written and read again
constexpr double kStream = 5.6e6;            // read once

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool widths_ok(const mok_fp8_shape *s) {
    return s && s->M >= 0 && s->N > 0 && s->K > 0 && s->N % 16 == 0 && s->K % 16 == 0 && s->N <= (1 << 20) &&
           s->K <= (1 << 20) && s->E >= 0 && s->E <= 4096 &&
           (s->out_dtype == MOK_STREAM_BF16 || s->out_dtype == MOK_STREAM_F32);
}

void fill(const mok_fp8_shape *s, BlkPlan *p) {
    *p = BlkPlan{};
    p->M = s->M;
    p->N = s->N;
    p->K = s->K;
    p->E = s->E;
    p->f32 = s->out_dtype == MOK_STREAM_F32;
    p->bm = 128;
    p->splits = 1;
}

double join_us(int runs, int64_t values) { return runs == 1 ? 0.0 : 5.0 + (double)runs * values * 8 / kTraffic; }

}  // namespace

mok_status make_blk_matmul_plan(const mok_fp8_shape *s, BlkPlan *p) {
    if (!widths_ok(s) || s->M >= (int64_t(1) << 31)) return MOK_ERROR_INVALID_VALUE;
    fill(s, p);
    const int64_t M = s->M, N = s->N, kb = ceil_div(s->K, 128), cols = ceil_div(N, 256);
    if ((ceil_div(M, 128) + s->E) * cols > kMostGroups) return MOK_ERROR_UNSUPPORTED;
    if (M == 0) return MOK_OK;
    // The experts' rows are not known here: taken as equal. Rows on one expert alone read one expert's weights, fewer
    // bytes in more passes: in us, equal / half of the rows on one / all on one, 16 experts x 8 rows x 7,168 x 2,048 (the
    // few-rows kernel) 40 / 50 / 30, 64 x 64 rows (tiles) 203 / 208 / 83, 16 x 32 rows x 4,096 x 7,168 91 / 125 / 46.
    const int64_t experts = s->E > 0 ? std::min<int64_t>(s->E, M) : 1, rows = ceil_div(M, experts);
    const double stream = (double)experts * N * s->K / kStream;   // the weights' bytes
    double least = 1e30;

    // 128-row tiles, the contraction in runs
    const int64_t tiles = experts * ceil_div(rows, 128) * cols;
    for (int r = 1; r <= kMostRuns && r <= kb; ++r) {
        const int64_t run = ceil_div(kb, r), groups = tiles * r;
        if (ceil_div(kb, run) != r) continue;
        if (r > 1 && (r * M * N * 4 > kPartBytes || (ceil_div(M, 128) + s->E) * cols * r > kMostGroups)) break;
        const double step = (groups <= 192 ? 0.83 : 0.95) * (p->f32 ? 1.8 : 1.0);
        const double us =
            5.0 + std::max(stream, (double)ceil_div(groups, kUnits) * (run * step + 1.0)) + join_us(r, M * N);
        if (us < least) {
            least = us;
            p->splits = r;
            p->run = (int)run;
        }
    }
    // 256-row tiles, with 128-row ones for an expert's last rows and the last round (bf16 results)
    if (!p->f32) {
        int64_t whole = experts * (rows / 256 + (rows % 256 > 128)) * cols;
        int64_t half = experts * (rows % 256 > 0 && rows % 256 <= 128 ? 1 : 0) * cols;
        if (whole % kUnits <= kUnits / 2) {
            half += whole % kUnits * 2;
            whole -= whole % kUnits;
        }
        half = std::max<int64_t>(half - (ceil_div(whole, kUnits) * kUnits - whole), 0);   // beside the last whole ones
        const double us = 5.0 + std::max(stream, (double)ceil_div(whole, kUnits) * (kb * 1.6 + 3.0) +
                                                     (double)ceil_div(half, kUnits) * (kb * 0.95 + 1.0));
        if (us < least) {
            least = us;
            p->bm = 256;
            p->splits = 1;
            p->run = 0;
        }
    }
    // 16 rows of the weights a workgroup, 16 mt rows at a time
    if (experts * N / 16 <= (1 << 22)) {
        // Two tiles of W a workgroup read X once for both and keep more loads in flight, where they still fill the
        // card. us with one and two: 64 x 7,168 x 2,048 13.2 / 10.4, 32 rows 9.0 / 7.6, 16 experts of one row 46 / 42,
        // of 8 rows 57 / 44; but 64 x 4,096 x 7,168 (128 workgroups) 24 / 30, one row 7.8 / 10.4.
        const int w = experts * (N / 32) >= 192 ? 2 : 1;
        // a pass is the weights' bytes, or its own latency; all rows of X come from L2 to every workgroup
        const double rate[3] = {w == 2 ? 30e6 : 12e6, 9e6, 6.5e6};
        for (int i = 0; i < 3; ++i) {
            const int64_t passes = ceil_div(rows, 16 << i);
            const double us =
                1.0 + (double)passes * std::max(stream, 2.5) + (double)M * (N / 16) * s->K / rate[i];
            if (us < least) {
                least = us;
                p->bm = 128;
                p->splits = 1;
                p->few = 1 << i;
                p->few_w = w;
            }
        }
    }
    if (p->splits > 1) p->total = (size_t)p->splits * M * N * 4;
    return MOK_OK;
}

// Weight gradients, us (rows, N x K of each expert; the choice marked *):
//                             256-row tiles   128-row tiles in 1 / 4 / 8 / 16 runs
//   512, 4,096 x 7,168        31*             35 / 242 / 448
//   8,192, 512 x 512          96              60 / 24 / 20.0 / 20.8 (13 runs: 20.6*)
//   1,024, 2,048 x 2,048      18              13.2* / 35 / 59
//   16,384 of 4, 2,048 x 1,024    57          43.7 - 46* / 95 / 149
//   8,192 of 16, 7,168 x 2,048    198*        253
// All of these are far from their floors (12.4, 1.7, 3.2, 25.6 and 105 us): a tile's stages fill a compute unit's LDS,
// so one workgroup runs on it and its fill, drain and store overlap with nothing.
mok_status make_blk_wgrad_plan(const mok_fp8_shape *s, BlkPlan *p) {
    if (!widths_ok(s) || s->M >= (int64_t(1) << 23) || s->M % 16) return MOK_ERROR_INVALID_VALUE;
    fill(s, p);
    const int64_t experts = std::max(s->E, 1), values = experts * s->N * s->K;
    const int64_t kb = std::max<int64_t>(ceil_div(ceil_div(s->M, 128), experts), 1);
    const auto groups = [&](int bm, int runs) {
        return (ceil_div(s->N, bm) * ceil_div(s->K, 256) * runs + 8) * experts;
    };
    if (groups(128, 1) > kMostGroups) return MOK_ERROR_UNSUPPORTED;
    double least = 1e30;
    for (int bm = 128; bm <= (p->f32 ? 128 : 256); bm *= 2) {
        const int64_t tiles = ceil_div(s->N, bm) * ceil_div(s->K, 256) * experts;
        for (int r = 1; r <= kMostRuns && r <= kb; ++r) {
            if (r > 1 && (r * values * 4 > kPartBytes || groups(bm, r) > kMostGroups)) break;
            const bool filled = tiles * r > 192;
            const double step = p->f32 ? 1.7 : bm == 128 ? (filled ? 1.1 : 0.92) : (filled ? 1.9 : 1.55);
            const double us = 5.0 + (double)ceil_div(tiles * r, kUnits) * (ceil_div(kb, r) * step + bm / 40.0) +
                              join_us(r, values);
            if (us < least) {
                least = us;
                p->bm = bm;
                p->splits = r;
            }
        }
    }
    if (p->splits > 1) p->total = (size_t)p->splits * values * 4;
    return MOK_OK;
}

}  // namespace mok
