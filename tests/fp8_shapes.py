"""Shapes at which the products on blocks of 128 take each of their paths: held to
fp64 on the GPU by test_gpu_fp8_tiles.py, and to the plan by test_fp8_plan.py."""

# M, N, K, fp32 result, what the plan takes: few (tiles of 16 rows), tile rows, runs
DENSE = {
    "few_1": (3, 4096, 1040, False, (1, 128, 1)),
    "few_2": (25, 4096, 2048, False, (2, 128, 1)),
    "few_4": (60, 1024, 1040, False, (4, 128, 1)),
    "few_4_two_passes": (100, 512, 272, False, (4, 128, 1)),
    "few_1_wide": (16, 6160, 1040, False, (1, 128, 1)),
    "few_2_wide": (25, 7184, 1040, False, (2, 128, 1)),              # 32 columns a workgroup, the last one 16
    "few_4_wide": (60, 6160, 2048, False, (4, 128, 1)),
    "few_4_wide_f32": (50, 7168, 1040, True, (4, 128, 1)),
    "few_2_wide_f32": (30, 6160, 272, True, (2, 128, 1)),
    "few_f32": (20, 1024, 4096, True, (2, 128, 1)),
    "runs": (128, 2064, 7168, False, (0, 128, None)),
    "runs_short_last": (300, 1040, 7088, False, (0, 128, None)),
    "runs_f32": (300, 1040, 7168, True, (0, 128, None)),
    "tiles_128": (900, 2064, 1040, False, (0, 128, 1)),
    "tiles_128_f32": (900, 2064, 1040, True, (0, 128, 1)),
    "halves_and_rest": (4400, 4096, 2048, False, (0, 256, 1)),      # 272 whole tiles: 256, 16 as halves, 16 for the rest
    "halves": (4500, 4112, 2048, False, (0, 256, 1)),               # 306 whole tiles: 256, 50 as halves, a narrow column
    "one_round": (3328, 4096, 2048, False, (0, 256, 1)),            # 208 whole tiles in one round
}

# rows of each expert, N, K, fp32 result, the plan's path
GROUPED = {
    "few": ([3, 0, 1, 7], 1024, 1040, False, (1, 128, 1)),
    "few_uneven": ([40, 0, 0, 2], 1024, 1040, False, (1, 128, 1)),   # three passes for one expert
    "few_1_wide": ([2, 0, 1, 16, 20], 2064, 1040, True, (1, 128, 1)),
    "few_wide": ([30, 0, 1, 40, 20], 2064, 1040, False, (2, 128, 1)),
    "runs": ([100, 0, 60, 30], 1040, 7168, False, (0, 128, None)),
    "tiles_128": ([130, 250, 0, 1, 380], 2064, 1040, False, (0, 128, 1)),
    "mixed": ([300, 0, 90, 1513, 256, 129, 2000, 512], 4096, 2048, False, (0, 256, 1)),
    "mixed_many": ([256] * 10 + [0, 255, 257, 128, 1] * 3 + [600] * 9, 2064, 2048, False, (0, 256, 1)),
}

# N, K, rows of each expert (None: one product of that many), fp32 result, tile rows, runs
WGRAD = {
    "whole": (4096, 7168, 512, False, (256, 1)),
    "runs": (512, 512, 8192, False, (128, None)),
    "runs_f32": (256, 528, 8192, True, (128, None)),
    "tiles_128": (1040, 1040, 1024, False, (128, 1)),
    "grouped_whole": (4096, 4112, [2048, 0, 128, 3408], False, (256, 1)),
    "grouped_runs": (256, 272, [3000, 0, 128, 5000], False, (128, None)),   # runs that stay empty for short experts
}
