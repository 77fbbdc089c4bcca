"""The kernels behind the products over groups of rows and the adapters, and for each sizes that reach it: run on the GPU by
test_gpu_routes.py, which asks the library for the kernel of every call, and held complete on the CPU by test_routes.py,
so that a change of a launch rule cannot leave a kernel without a test."""

# bsm_gemm_grouped: kernel -> [(rows of the groups, N, K)]; B_k and B_n where the kernel takes both orders.
# Groups end in tiles of up to 32, 64, 128 and more rows; K below a tile, of whole tiles, and of tiles and a rest.
RAGGED = [33, 130, 257, 300, 64, 97, 1, 0, 170, 31, 128, 65]
GROUPED = {
    "k_grouped_skinny<1>": [([16, 1, 0, 7], 50, 500)],
    "k_grouped_skinny<2>": [([30, 20, 33], 50, 500)],
    "k_grouped_skinny<4>": [([60, 1, 64, 50], 50, 500)],
    "k_grouped_split": [([100, 90, 40, 65], 260, 200)],
    "k_grouped_mid": [(RAGGED, 1601, 40), (RAGGED, 1601, 200), (RAGGED, 1601, 1000)],
    "k_grouped": [([1300, 770, 3, 2047], 4100, 200)],
}
K_MAJOR_ONLY = ("k_grouped_skinny<1>", "k_grouped_skinny<2>", "k_grouped_skinny<4>")

# bsm_gemm_grouped_wgrad: kernel -> [(rows of the groups, M, N)]
WGRAD = {
    "k_grouped_wgrad<256, 32, 2, 1>": [([400, 0, 1030, 35], 1300, 2820)],
    "k_grouped_wgrad<128, 64, 1, 2>": [([1500, 0, 1663], 200, 140)],
    "k_grouped_wgrad<128, 32, 4, 1>": [([5, 0, 64, 31, 130], 300, 520)],
    "k_grouped_wgrad<128, 64, 2, 1>": [([255, 256, 257], 300, 520)],
}

# bsm_gemm_grouped_block_scale: kernel -> (pairs (A, B, fast), [(rows of the groups, N, K)])
PAIRS = [("e4m3", "e4m3", 0), ("e4m3", "e4m3", 1), ("e4m3", "e2m1", 0), ("e4m3", "e2m1", 1), ("e2m1", "e2m1", 0), ("e2m1", "e2m1", 1)]
GENERAL = [("e4m3", "e4m3", 0), ("e4m3", "e2m1", 0), ("e4m3", "e2m1", 1)]
FEW = [33, 130, 170, 64, 97, 1, 0, 128, 65, 100, 40, 31]
LONG = [700, 300, 3, 520]
MX = {
    "k_grouped_mx_split": (PAIRS, [([70, 15, 16, 33], 260, 1184)]),
    "k_grouped_mx_rows32": ([("e4m3", "e2m1", 0)], [([(7 * i) % 9 for i in range(40)] + [70, 0, 33], 1300, 1184)]),
    "k_grouped_mx_mid": (PAIRS, [(FEW, 2001, 96), (FEW, 2001, 160), (FEW, 2001, 1184)]),
    "k_gemm_mx": ([p for p in PAIRS if p not in GENERAL], [(LONG, 4100, 1184)]),
    "k_gemm_mx_any": (GENERAL, [(LONG, 4100, 1184)]),
}

# bsm_gemm_lora: (kernel of the projection, of the shrink) -> [(rows, N, K, R, adapters)]
LORA = {
    ("k_lora_skinny<1>", "k_lora_shrink_rows"): [(15, 136, 200, 16, 7)],
    ("k_lora_skinny<2>", "k_lora_shrink_rows"): [(31, 136, 200, 40, 7)],
    ("k_lora_skinny<3>", "k_lora_shrink_rows"): [(47, 136, 200, 16, 7)],
    ("k_lora_skinny<4>", "k_lora_shrink_rows"): [(63, 136, 200, 16, 7), (200, 136, 520, 12, 5)],
    ("k_lora_skinny<4>", "k_lora_shrink"): [(1000, 250, 520, 130, 8)],
    ("k_lora<2>", "k_lora_shrink_rows"): [(200, 1500, 264, 24, 3)],
    ("k_lora<2>", "k_lora_shrink"): [(1100, 1100, 264, 72, 3)],
    ("k_lora<1>", "k_lora_shrink_rows"): [(2900, 1100, 200, 24, 40)],
    ("k_lora<1>", "k_lora_shrink"): [(3300, 1100, 200, 130, 3)],
    ("k_lora<1>", ""): [(3300, 1100, 200, 0, 3)],
}
