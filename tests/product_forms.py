"""Products that reach every kernel of the MXFP4 products and of their gradient:
(kernel, kind of rows or "dx", rows of each expert, n, k, rows of no expert,
rows to gather from).  tests/test_operator_launches.py holds each to its kernel,
tests/test_gpu_mxfp4_forms.py runs it."""

# runs of 256 rows and of every class of rest: up to 16, 32, 64, 96, 128, 192, 256
RUNS = [300, 0, 500, 290, 129, 170, 200, 257, 511, 640, 33, 193, 192, 800, 70, 100, 20]
MIDDLE = [64, 3, 17, 33, 0, 130, 100, 81]                     # runs of 64 rows, rests of each class
THIN = [1, 0, 2, 16, 9, 17, 5, 7]                             # units of 16 rows
FEW = [13 if i % 8 == 3 else i % 4 for i in range(64)]        # under four rows per expert
ONES, MANY_ONES = [1] * 8, [1] * 128
FAR = 2_100_000                                               # rows whose bytes pass 32-bit offsets

PRODUCTS = [
    # few rows: 16, 32 and 64 outputs; rows in LDS throughout, and in slabs (of 1024
    # inputs for 9 to 16 rows, of 2048 for 7, of three times 1024 for 5); blocks in pairs or an odd number
    ("mx_matmul_thin<false, 1, false>", "bf16", THIN, 65, 96, 1, 0),
    ("mx_matmul_thin<false, 1, false>", "bf16", THIN, 30, 3232, 0, 30),
    ("mx_matmul_thin<false, 1, true>", "bf16", THIN, 64, 2112, 0, 30),
    ("mx_matmul_thin<false, 2, false>", "bf16", ONES, 2050, 2080, 0, 1),
    ("mx_matmul_thin<false, 2, true>", "bf16", ONES, 2050, 2112, 0, 1),
    ("mx_matmul_thin<false, 4, false>", "bf16", FEW, 1001, 1056, 1, 40),
    ("mx_matmul_thin<false, 4, true>", "bf16", FEW, 1001, 1088, 1, 0),
    ("mx_matmul_thin<true, 1, false>", "mxfp4", THIN, 65, 96, 1, 0),
    ("mx_matmul_thin<true, 1, true>", "mxfp4", THIN, 64, 2112, 0, 30),
    ("mx_matmul_thin<true, 2, false>", "mxfp4", ONES, 2050, 2080, 0, 1),
    ("mx_matmul_thin<true, 2, true>", "mxfp4", ONES, 2050, 2112, 0, 1),
    ("mx_matmul_thin<true, 4, false>", "mxfp4", FEW, 1001, 1056, 1, 40),
    ("mx_matmul_thin<true, 4, true>", "mxfp4", FEW, 1001, 1088, 1, 0),
    # two tiles to a workgroup: an odd and an even number of tiles, with and without slabs
    ("mx_matmul_thin<false, 4, false>", "bf16", MANY_ONES, 4033, 96, 1, 0),
    ("mx_matmul_thin<false, 4, true>", "bf16", MANY_ONES, 4100, 128, 0, 9),
    ("mx_matmul_thin<false, 4, false>", "bf16", [700, 900, 400], 4150, 1056, 0, FAR),
    ("mx_matmul_thin<false, 4, true>", "bf16", [700, 900, 400], 4150, 1088, 0, FAR),
    ("mx_matmul_thin<true, 4, false>", "mxfp4", MANY_ONES, 4033, 96, 1, 0),
    ("mx_matmul_thin<true, 4, true>", "mxfp4", MANY_ONES, 4100, 128, 0, 9),
    # 64 rows x 128 outputs: scales by groups (k a multiple of 128) and by bytes
    ("mx_matmul_mid<true>", "bf16", MIDDLE, 701, 128, 0, 0),
    ("mx_matmul_mid<true>", "bf16", MIDDLE, 701, 1152, 1, 77),
    ("mx_matmul_mid<false>", "bf16", MIDDLE, 701, 1056, 0, 77),
    ("mx_matmul_mid<true>", "bf16", [500], 1001, 640, 0, 0),
    # 256 x 256
    ("mx_matmul_large<true>", "bf16", RUNS, 2555, 128, 0, 77),
    ("mx_matmul_large<true>", "bf16", RUNS, 2555, 640, 1, 0),
    ("mx_matmul_large<false>", "bf16", RUNS, 2555, 672, 1, 77),
    ("mx_matmul_large<true>", "bf16", [4100], 2700, 256, 0, 0),
    # 256 x 256, both sides in 4 bits: one, two, three and more stages; groups of scales that
    # end in the middle
    ("mx_matmul4<true>", "mxfp4", RUNS, 260, 256, 1, 0),
    ("mx_matmul4<true>", "mxfp4", RUNS, 260, 512, 0, 77),
    ("mx_matmul4<true>", "mxfp4", RUNS, 300, 768, 3, 0),
    ("mx_matmul4<true>", "mxfp4", RUNS, 300, 1280, 0, 77),
    ("mx_matmul4<true>", "mxfp4", RUNS, 257, 2048, 0, 0),
    ("mx_matmul4<true>", "mxfp4", [300], 4100, 1536, 0, 0),
    ("mx_matmul4<false>", "mxfp4", RUNS, 260, 32, 1, 0),
    ("mx_matmul4<false>", "mxfp4", RUNS, 300, 1056, 0, 77),
    # gradient, few rows: fewer and more than 128 workgroups, one and several steps per wave
    ("mx_matmul_dx_thin<1, 8>", "dx", THIN, 32, 160, 1, 0),
    ("mx_matmul_dx_thin<1, 8>", "dx", THIN, 544, 160, 1, 0),
    ("mx_matmul_dx_thin<2, 4>", "dx", [1, 2, 0] * 14, 64, 1056, 1, 0),
    ("mx_matmul_dx_thin<2, 4>", "dx", [1, 2, 0] * 14, 544, 1056, 1, 0),
    ("mx_matmul_dx_thin<2, 4>", "dx", FEW, 288, 544, 0, 0),
    # gradient, 64 rows x 256 columns, and 256 x 256: one to many stages
    ("mx_matmul_dx_mid", "dx", [250, 1, 300, 64, 0, 885], 64, 1440, 0, 0),
    ("mx_matmul_dx_mid", "dx", [250, 1, 300, 64, 0, 885], 352, 1440, 1, 0),
    ("mx_matmul_dx_fat", "dx", RUNS, 32, 2528, 0, 0),
    ("mx_matmul_dx_fat", "dx", RUNS, 192, 2528, 1, 0),
    ("mx_matmul_dx_fat", "dx", RUNS, 416, 2528, 1, 0),
    ("mx_matmul_dx_fat", "dx", [4100], 160, 2720, 0, 0)]

NAMES = [f"{kind}-{i}-{kernel.split('_')[-1]}" for i, (kernel, kind, *_) in enumerate(PRODUCTS)]
