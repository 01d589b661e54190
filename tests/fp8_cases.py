"""Shapes of FP8 products over every tile of the persistent kernel, with more
tiles than workgroups, ragged edges and four to seven blocks of 128 contracted
channels (each a phase of its ring of five units). test_fp8_dispatch.py holds
the library's choice to them, test_gpu_fp8_tiles.py the results."""

# (rows, columns): {tile}
OUTPUTS = {(256, 256): (4592, 12272), (256, 192): (2100, 8208), (128, 128): (32800, 272)}
# (rows, columns) of a weight gradient, both multiples of 16
GRADIENTS = {(256, 256): (12272, 4592), (256, 192): (8208, 2096), (128, 128): (32800, 272)}
CONTRACTED = {4: 400, 5: 528, 6: 768, 7: 784}   # blocks: channels (K % 16 == 0)
TOKENS = {4: 450, 5: 600, 6: 768, 7: 777}       # blocks: tokens of a weight gradient

FORWARD = [(tile, blocks, m, CONTRACTED[blocks], n) for tile, (m, n) in OUTPUTS.items() for blocks in CONTRACTED]
BACKWARD = [(tile, blocks, TOKENS[blocks], k, n) for tile, (n, k) in GRADIENTS.items() for blocks in TOKENS]

# large inputs: more than 16 MB to quantize; more than 128 MB of x, dy and dx, which the norm's gradients read past the caches
QUANTIZED = [(4099, 2064), (9001, 912)]                    # rows, channels
NORM_GRADIENTS = [(10600, 2051, "bf16"), (8600, 1283, "fp32"), (3700, 6001, "fp16")]
