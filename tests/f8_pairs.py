"""Sizes (M, N, K) of the 8-bit floating-point product that its planner gives to pairs of blocks on 152 SMs, and
ones that it gives to the other form.  Checked on the CPU by test_ssm_forms.py, run on the GPU by
test_gpu_f8_pairs.py."""
SMS = 152
PAIRS = [
    (2000, 2040, 300),    # one tile a pair, three steps: fewer than the ring's stages; ragged in M, N and K
    (1100, 2101, 1024),   # rows of y off 16 bytes
    (2048, 2048, 2048),   # nothing ragged; the ring goes round
    (1300, 4100, 1160),   # more tiles than pairs: two rounds
    (4096, 2048, 640),    # weight gradients' shape
]
EXACT = (1100, 2100, 640)
STRIDED = (1100, 2100, 520)
CALLS = [(1100, 2100, 1024), (1300, 4100, 1160), (2048, 2048, 512), (1100, 2100, 520)]
OTHERS = [(600, 1000, 1024), (3, 256, 4096), (197, 500, 2000)]
