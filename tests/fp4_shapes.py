"""Product shapes that reach each MXFP4 kernel, and which one: what
mlpblk_fp4_product_kernel answers for them, checked on the host and before each GPU test
that relies on it, so that a change of the rule cannot move a test off its kernel unseen.

Kernels: "tma" and "pair" (CTA pairs, C stored by TMA or by threads), or the number of CTAs
that share a tile's K."""

# (m, n, k), out, accumulate, kernel
DENSE = [
    ((2500, 2600, 1600), "bf16", False, "tma"), ((2500, 2600, 1600), "f32", False, "tma"),
    ((2500, 2600, 1600), "f32", True, "tma"), ((2500, 2601, 320), "bf16", False, "pair"),
    ((2305, 2311, 1600), "f32", False, "pair"), ((2305, 2311, 1600), "f32", True, "pair"),
    ((2305, 2310, 1600), "f32", True, "pair"), ((2049, 1304, 4100), "bf16", False, "tma"),
    ((1030, 1100, 520), "f32", True, 1), ((333, 1001, 1031), "bf16", False, 1),
    # K split over 2, 4 and 8 CTAs
    ((700, 1280, 10300), "f32", False, 2), ((700, 1279, 10300), "f32", True, 2), ((700, 1280, 10300), "bf16", False, 2),
    ((300, 1270, 10300), "f32", True, 4), ((300, 1271, 10300), "bf16", False, 4),
    ((3, 300, 8192), "f32", True, 8), ((200, 128, 16384), "f32", True, 8), ((200, 130, 16384), "f32", False, 8),
    ((1, 1025, 9000), "bf16", False, 8), ((33, 257, 12000), "f32", True, 8),
]

# (T, d, n, E, k, pad), out, accumulate, kernel: matmul_grouped of T tokens' top-k rows
GROUPED = [
    ((3000, 1300, 1001, 5, 2, 128), "f32", False, "pair"), ((3000, 1300, 1001, 5, 2, 128), "f32", True, "pair"),
    ((3000, 136, 1001, 5, 2, 256), "bf16", False, "pair"), ((3000, 136, 1000, 5, 2, 128), "f32", True, "tma"),
    ((900, 4200, 1200, 4, 2, 128), "bf16", False, "tma"),
    ((20, 10300, 300, 3, 2, 128), "bf16", False, 8), ((20, 10300, 301, 3, 2, 128), "f32", False, 8),
    ((20, 10300, 300, 3, 2, 256), "f32", True, 8), ((150, 10400, 600, 4, 2, 128), "f32", True, 2),
]

# (T, d, n, E, k), accumulate, kernel: wgrad_grouped C[E][n, d]
WGRAD = [
    ((4000, 1023, 1200, 6, 2), False, "pair"), ((4000, 1023, 1200, 6, 2), True, "pair"),
    ((4000, 1020, 1200, 6, 2), True, "tma"),
    ((5200, 200, 100, 4, 2), False, 8), ((5200, 200, 100, 4, 2), True, 8), ((5200, 201, 30, 4, 2), True, 8),
    ((5200, 500, 300, 4, 2), True, 2),
]


def dense_desc(mb, shape, out, accumulate):
    return mb.make_fp4_matmul_desc(*shape, out, accumulate)


def grouped_desc(mb, case, out, accumulate):
    T, d, n, E, k, pad = case
    R = mb.mlpblk_moe_sort_rows(mb.make_sort_desc(T, d, E, k, pad))
    return mb.make_fp4_matmul_desc(R, n, d, out, accumulate, E, pad, T * k)


def wgrad_desc(mb, case, accumulate):
    T, d, n, E, k = case
    R = mb.mlpblk_moe_sort_rows(mb.make_sort_desc(T, d, E, k, 256))
    return mb.make_fp4_matmul_desc(n, d, R, "f32", accumulate, E, 256)


def kernel(mb, desc, form, sms):
    r = mb.mlpblk_fp4_product_kernel(desc, form, sms)
    return {mb.MLPBLK_FP4_KERNEL_PAIR_TMA: "tma", mb.MLPBLK_FP4_KERNEL_PAIR: "pair"}.get(r, r)
