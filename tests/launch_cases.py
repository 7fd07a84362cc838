"""Calls of the row operators whose kernels take 1024 lanes a row, with more rows
than one launch takes: 2^31 work items, so 2^21 rows."""
LAUNCH_ROWS = 1 << 21
# operator, columns (of SwiGLU: of its result), type of the result
CASES = [("rmsnorm", 16392, "bf16"), ("rmsnorm", 16392, "e4m3"), ("rmsnorm", 32776, "mxfp4"), ("swiglu", 12296, "e4m3"),
         ("swiglu", 16392, "e4m3")]
