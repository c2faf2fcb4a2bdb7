"""Shapes of the recurrence that take each of its kernels, with what the split rule
makes of them.  test_recurrence_paths.py holds the rule to it on the CPU,
test_gpu_recurrence_paths.py runs them."""

# (types, batch, time, channels): per direction (bytes of a row, frames of a lane, time
# ranges, tiles of a range)
PATHS = [
    # 64-byte rows, whose workgroups are reordered by pairs; whole tiles, a last one in part
    (("f16", "bf16"), (8, 700, 1000), (64, 4, 1, 3), (128, 2, 4, 3)),
    (("f16", "bf16"), (8, 700, 1021), (64, 4, 1, 3), (128, 2, 4, 3)),
    (("f32",), (6, 600, 1000), (64, 2, 1, 3), (64, 2, 1, 3)),
    (("f32",), (6, 600, 1021), (64, 2, 1, 3), (64, 2, 1, 3)),
    # a number of workgroups that is no multiple of 16
    (("f16", "bf16"), (9, 600, 610), (64, 4, 1, 3), (128, 2, 5, 2)),
    (("f32",), (11, 800, 250), (64, 2, 1, 4), (64, 2, 1, 4)),
    # 128-byte rows, several whole tiles in one walk
    (("f16", "bf16"), (260, 800, 64), (128, 4, 1, 7), (128, 2, 1, 13)),
    (("f16", "bf16"), (130, 800, 125), (128, 4, 1, 7), (128, 2, 1, 13)),
    (("f32",), (130, 800, 64), (128, 4, 1, 4), (128, 2, 1, 7)),
    (("f32",), (130, 800, 61), (128, 4, 1, 4), (128, 2, 1, 7)),
    # time ranges of several tiles each
    (("f16", "bf16"), (60, 3000, 64), (128, 4, 8, 3), (128, 2, 8, 6)),
    (("f16", "bf16"), (30, 3001, 77), (128, 4, 8, 3), (128, 2, 8, 6)),
    (("f32",), (30, 6000, 61), (128, 4, 8, 3), (128, 2, 8, 6)),
]
