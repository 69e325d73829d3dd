"""Sizes of the product under the adapters' calls, with the plan that each is for:
test_lora_plan.py asks the library's plan on the CPU (for 256 compute units),
test_gpu_lora_paths.py runs them, forward (y [M][out]) and backward (dx [M][out])."""

# M, out, contraction, fast -> (tile rows, tile columns, K parts, rows of a head launch, is it
# the fast products' own 256 x 256 kernel)
PATHS = {
    "fast 256x256": ((3900, 3896, 1500, True), (256, 256, 1, 0, True)),
    "fast 256x256, odd rows of the result": ((3900, 3901, 1500, True), (256, 256, 1, 0, True)),
    "fast 256x256, last tiles in K parts": ((2251, 1812, 6703, True), (256, 256, 3, 0, True)),
    "fast 128x128": ((3900, 3896, 200, True), (128, 128, 1, 0, False)),
    "fast 128x64 in K parts": ((2100, 150, 6000, True), (128, 64, 5, 0, False)),
    "fast 64x128 in K parts": ((150, 2100, 6000, True), (64, 128, 5, 0, False)),
    "fast 64x64 in K parts": ((300, 264, 4000, True), (64, 64, 8, 0, False)),
    "fast 64x64": ((333, 1500, 4000, True), (64, 64, 1, 0, False)),
    "binary32 256x256": ((3900, 3896, 200, False), (256, 256, 1, 0, False)),
    "binary32 256x256 in K parts": ((1675, 2432, 4973, False), (256, 256, 3, 0, False)),
    "binary32 256x256 and a tail": ((16500, 4000, 300, False), (256, 256, 1, 16384, False)),
    "binary32 128x128 in K parts": ((700, 2100, 8000, False), (128, 128, 2, 0, False)),
    "binary32 128x64 in K parts": ((2100, 150, 6000, False), (128, 64, 5, 0, False)),
    "binary32 64x128 in K parts": ((150, 2100, 6000, False), (64, 128, 5, 0, False)),
    "binary32 64x64 in K parts": ((300, 264, 4000, False), (64, 64, 8, 0, False)),
    "binary32 64x64": ((333, 1500, 4000, False), (64, 64, 1, 0, False)),
}
