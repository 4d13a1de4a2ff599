"""Products that take every form of the free products' kernels, dense and over
ragged groups: what the GPU tests run, and the CPU tests hold to the rule."""
import torch

import combine_router_gemm_softmax_b200 as M

BF16, F32 = torch.bfloat16, torch.float32
FEW, SINGLE, PAIR, SPLIT = M.MOE_FORM_FEW_ROWS, M.MOE_FORM_SINGLE, M.MOE_FORM_PAIR, M.MOE_FORM_SPLIT

# (product, type, rows of each group (one number: a dense product), n, k, padding of the rows, form, columns of a tile)
FORMS = [
    # few rows: 16 features a CTA, 32 in eight warps, 32 in four; reductions of an odd length and of several chains
    ("forward", BF16, 7, 136, 136, 0, FEW, 0), ("forward", BF16, 8, 6000, 1001, 8, FEW, 0),
    ("forward", BF16, 5, 16000, 264, 0, FEW, 0), ("forward", BF16, 3, 9600, 17000, 0, FEW, 0),
    ("forward", BF16, [2, 0, 9, 1], 136, 264, 0, FEW, 0), ("forward", BF16, [300, 0, 31, 8], 16, 520, 0, FEW, 0),
    ("forward", BF16, 331, 520, 136, 0, SINGLE, 64), ("forward", BF16, 777, 4096, 136, 0, SINGLE, 224),
    ("forward", BF16, [13, 0, 40], 2048, 136, 0, SINGLE, 64), ("forward", BF16, [500, 129, 0, 655], 2043, 136, 8, SINGLE, 192),
    ("forward", BF16, 12293, 136, 2048, 0, PAIR, 160), ("forward", BF16, 12293, 519, 1031, 8, PAIR, 192),
    ("forward", BF16, [600, 0, 1, 1033, 2048, 409], 136, 4096, 0, PAIR, 64),
    ("forward", BF16, [4100, 0, 8188], 520, 136, 0, PAIR, 256),
    ("forward", BF16, 777, 136, 2048, 0, SPLIT, 64), ("forward", BF16, 331, 4096, 4096, 0, SPLIT, 192),
    ("forward", BF16, [70, 0, 200, 1, 33, 19], 264, 2047, 8, SPLIT, 64),
    ("dgrad", BF16, 7, 136, 136, 0, SINGLE, 64), ("dgrad", BF16, 2051, 135, 1031, 8, SINGLE, 192),
    ("dgrad", BF16, [3, 0, 130], 136, 520, 0, SINGLE, 64), ("dgrad", BF16, [50, 0, 9, 200, 1, 63], 136, 4096, 0, SINGLE, 192),
    ("dgrad", BF16, 16381, 1032, 136, 0, PAIR, 128), ("dgrad", BF16, 8209, 263, 4091, 8, PAIR, 256),
    ("dgrad", BF16, [12000, 1, 0, 260, 17, 7], 1032, 136, 0, PAIR, 128), ("dgrad", BF16, [8000, 4285, 0], 136, 520, 0, PAIR, 256),
    ("dgrad", BF16, 7, 2048, 136, 0, SPLIT, 64), ("dgrad", BF16, 2051, 4096, 520, 0, SPLIT, 192),
    ("dgrad", BF16, [130, 0, 7], 2048, 135, 8, SPLIT, 64), ("dgrad", BF16, [300, 0, 1, 255, 150, 60], 4096, 1032, 0, SPLIT, 192),
    # weight gradients: rows next to the 16 of an MMA, the 64 of a block and the 512 of an accumulator
    ("wgrad", BF16, 7, 136, 136, 0, SINGLE, 64), ("wgrad", BF16, 513, 1400, 4091, 8, SINGLE, 192),
    ("wgrad", BF16, [0, 512, 511, 1, 513, 65, 0], 264, 1032, 0, SINGLE, 192),
    ("wgrad", BF16, 4099, 4096, 1032, 0, PAIR, 128), ("wgrad", BF16, 8191, 4096, 4096, 0, PAIR, 256),
    ("wgrad", BF16, 8193, 4091, 4090, 8, PAIR, 256), ("wgrad", BF16, 512 * 17 + 31, 4096, 4096, 0, PAIR, 256),
    ("wgrad", BF16, [12279, 12285], 2048, 1032, 0, PAIR, 128), ("wgrad", BF16, [18000, 14742], 1543, 519, 8, PAIR, 128),
    ("wgrad", BF16, 2051, 136, 136, 0, SPLIT, 64), ("wgrad", BF16, 2051, 519, 2047, 8, SPLIT, 192),
    ("wgrad", BF16, [6100, 0, 49], 136, 136, 0, SPLIT, 64), ("wgrad", BF16, [2049, 1, 4099], 264, 1032, 0, SPLIT, 192),
    # fp32: few rows by one, two and four tokens; 64 and 128 wide tiles, reductions in clusters
    ("forward", F32, 1, 136, 1030, 0, FEW, 0), ("forward", F32, 2, 51, 264, 1, FEW, 0), ("forward", F32, 7, 136, 136, 0, FEW, 0),
    ("forward", F32, 6157, 136, 136, 0, SINGLE, 64), ("forward", F32, 12293, 135, 136, 1, SINGLE, 128),
    ("forward", F32, [600, 0, 1, 400, 280, 7], 520, 136, 0, SINGLE, 64), ("forward", F32, [9, 0, 40, 1, 3, 0], 4096, 135, 1, SINGLE, 128),
    ("forward", F32, 61, 136, 136, 0, SPLIT, 64), ("forward", F32, [30, 0, 23], 136, 2051, 1, SPLIT, 64),
    ("dgrad", F32, 6157, 136, 136, 0, SINGLE, 64), ("dgrad", F32, 12293, 135, 136, 1, SINGLE, 128),
    ("dgrad", F32, [600, 0, 1, 400, 280, 7], 136, 520, 0, SINGLE, 64), ("dgrad", F32, [0, 3, 1, 0, 2, 1], 135, 4096, 1, SINGLE, 128),
    ("dgrad", F32, 7, 136, 136, 0, SPLIT, 64), ("dgrad", F32, [3, 0, 130], 1030, 135, 1, SPLIT, 64),
    ("wgrad", F32, 7, 136, 136, 0, SINGLE, 64), ("wgrad", F32, 7, 519, 4096, 1, SINGLE, 128),
    ("wgrad", F32, [3, 0, 2], 136, 136, 0, SINGLE, 64), ("wgrad", F32, [700, 0, 33, 1, 2, 64], 520, 519, 1, SINGLE, 128),
    ("wgrad", F32, 20011, 136, 136, 0, SPLIT, 64), ("wgrad", F32, [300, 0, 15000], 136, 135, 1, SPLIT, 64),
]
# bf16 reductions of several accumulators: (rows of each group, length, width, the forward's form, the input gradient's)
LONG = [
    ([4], 1 << 20, 16, FEW, SPLIT), ([3], (1 << 16) + 24, 9600, FEW, SPLIT), ([300], (1 << 19) + 8, 264, SPLIT, SPLIT),
    ([2048], 1 << 17, 2048, PAIR, PAIR), ([200, 0, 130, 7, 500], (1 << 18) + 72, 328, SPLIT, SPLIT),
    ([16384], 3 * 16384 + 64, 136, PAIR, PAIR), ([500, 0, 300, 129, 7, 255, 400, 409], 16384 + 64, 4096, SINGLE, SINGLE),
]
FIRST, LAST = 3, 5  # rows of a ragged buffer before its first group and after its last


def rows_of(sizes):
    """Rows of a case's buffers."""
    return sizes if isinstance(sizes, int) else sum(sizes) + FIRST + LAST


def form_of(case, sms):
    product, dt, sizes, n, k = case[:5]
    return M.moe_product_form_used(product, rows_of(sizes), n, k, 1 if isinstance(sizes, int) else len(sizes), dt, sms)


def name_of(case):
    product, dt, sizes, n, k, _, form, bn = case
    groups = "dense" if isinstance(sizes, int) else f"{len(sizes)}groups"
    return f"{product}-{'bf16' if dt == BF16 else 'f32'}-{groups}-{rows_of(sizes)}x{n}x{k}-{['few', 'single', 'pair', 'split'][form]}{bn}"
