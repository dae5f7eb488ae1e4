"""Bounds that give each kernel of q8_attention_kv8_tree its calls: rows of a workgroup (16 and 32 that its
waves take for themselves, 128 or 256 that share codes in LDS) and whether the keys are split.  The data of a
call may be far smaller than its bounds; test_tree_kernels.py holds the rows against the rule."""

# name: (rows of a workgroup, split, seqs, heads, kv_heads, dim, page, max_q, max_kv, window)
KERNELS = {
    "16 rows, 64": (16, False, 3, 4, 2, 64, 32, 40, 1000, 0),
    "16 rows, 64, split": (16, True, 3, 4, 2, 64, 64, 40, 30000, 0),
    "16 rows, 128": (16, False, 3, 4, 2, 128, 64, 40, 1000, 0),
    "16 rows, 128, split": (16, True, 2, 4, 2, 128, 128, 16, 30000, 0),
    "16 rows, 256": (16, False, 3, 4, 2, 256, 32, 40, 500, 0),
    "16 rows, 256, split": (16, True, 3, 4, 2, 256, 128, 40, 30000, 0),
    "32 rows": (32, False, 64, 32, 8, 128, 32, 6, 700, 0),
    "32 rows, split": (32, True, 2, 8, 2, 128, 64, 16, 60000, 0),
    "shared, 64": (256, False, 3, 16, 2, 64, 32, 4000, 9000, 40),
    "shared, 64, split": (256, True, 2, 8, 2, 64, 64, 64, 100000, 0),
    "shared, 64, window": (256, True, 20, 4, 1, 64, 128, 64, 30000, 20000),
    "shared, 128": (256, False, 3, 16, 2, 128, 64, 2000, 9000, 40),
    "shared, 128, split": (256, True, 2, 8, 2, 128, 32, 64, 100000, 0),
    "shared, 128, window": (256, True, 10, 4, 1, 128, 128, 64, 30000, 20000),
    "shared, 256": (128, False, 3, 16, 2, 256, 128, 1500, 9000, 40),
    "shared, 256, split": (128, True, 2, 4, 1, 256, 64, 32, 100000, 0),
    "shared, 256, window": (128, True, 10, 4, 1, 256, 32, 32, 30000, 20000),
}
