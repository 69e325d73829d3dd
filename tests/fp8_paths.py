"""Sizes that reach the 8-bit operators' paths of large or split products, with the plan
that each is for: test_fp8_plan.py asks the library's plan on the CPU (for 256 compute
units), test_gpu_fp8_paths.py runs them."""

# M, N, K, fast -> (tile rows, tile columns, K parts, rows of a head launch, is it the fast
# products' own 256 x 256 kernel)
PRODUCTS = {
    "binary32 256x256, aligned rows of C": ((3900, 3896, 1500, False), (256, 256, 1, 0, False)),
    "binary32 256x256, odd rows of C": ((3900, 3901, 1500, False), (256, 256, 1, 0, False)),
    "binary32 256x256 and a tail, aligned": ((16500, 4000, 700, False), (256, 256, 1, 16384, False)),
    "binary32 256x256 and a tail, odd": ((16500, 4001, 700, False), (256, 256, 1, 16384, False)),
    "binary32 256x256 in K parts": ((4100, 1030, 12300, False), (256, 256, 3, 0, False)),
    "binary32 128x128": ((4200, 4000, 700, False), (128, 128, 1, 0, False)),
    "binary32 64x128": ((136, 10000, 3000, False), (64, 128, 1, 0, False)),
    "binary32 128x64": ((10000, 136, 3000, False), (128, 64, 1, 0, False)),
    "binary32 32x128 in K parts": ((31, 300, 2000, False), (32, 128, 4, 0, False)),
    "binary32 16x128 in K parts": ((5, 4100, 4090, False), (16, 128, 7, 0, False)),
    "fast 256x256, aligned rows of C": ((3900, 3896, 1500, True), (256, 256, 1, 0, True)),
    "fast 256x256, odd rows of C": ((3900, 3901, 1500, True), (256, 256, 1, 0, True)),
    "fast 256x256, last tiles in K parts": ((4300, 3900, 4000, True), (256, 256, 8, 0, True)),
    "fast 64x128": ((4200, 4001, 700, True), (64, 128, 1, 0, False)),
    "fast 128x64": ((10000, 136, 1500, True), (128, 64, 1, 0, False)),
    "fast 128x128": ((1500, 3000, 3000, True), (128, 128, 1, 0, False)),
    "fast 32x128": ((17, 129, 640, True), (32, 128, 1, 0, False)),
    "fast 16x128 in K parts": ((5, 4100, 4090, True), (16, 128, 7, 0, False)),
}

# M, K, F, fast -> the forward pass's first half: "fused" (one kernel), "dual" with K parts,
# or "apart" (two products, then the activation); the dual product's tile rows where named
FORWARD = {
    "fast, one kernel": ((2500, 130, 4000, True), ("fused", 1)),
    "fast, dual in K parts": ((8, 4096, 384, True), ("dual", 8)),
    "fast, dual in one part": ((300, 300, 1100, True), ("dual", 1)),
    "binary32, dual in K parts": ((8, 4096, 384, False), ("dual", 8)),
    "binary32, dual of 256x256 tiles": ((150, 4600, 24740, False), ("dual", 1, 256)),
    "binary32, apart": ((4100, 1030, 6100, False), ("apart", 1)),
}

# M, K, F, fast -> dx's plan as above (both terms, one after the other in K), whether dh and
# its step are one kernel, and the three weight gradients' launch: (K parts of the last
# tiles, unsplit tiles), or None where each has its own
BACKWARD = {
    "fast, dx of the 256x256 kernel in K parts": ((4100, 1030, 6100, True), (256, 256, 3, 0, True), False, None),
    "fast, dx of the 256x256 kernel": ((3900, 3896, 800, True), (256, 256, 1, 0, True), False, None),
    "fast, gradients in one launch with K parts": ((4096, 1024, 6144, True), (64, 128, 1, 0, False), True, (8, 256)),
    "binary32, dx of 256x256 tiles in K parts": ((4100, 1030, 6100, False), (256, 256, 3, 0, False), False, None),
    "binary32, dx of 256x256 tiles": ((3900, 3896, 800, False), (256, 256, 1, 0, False), False, None),
}
