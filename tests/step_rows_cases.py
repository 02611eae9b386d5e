"""Sizes at which a thread of the single-token state update has two or four rows and the
division leaves something over: rows past the head's last, vectors that overlap the one
before, lanes past the row, workgroups of fewer waves.  Shared by the GPU test that runs
them and the CPU test that holds them to the rows they are meant to have."""

CASES = {
    # rows per thread, (batch, H, P, N, G, dtype, dt dtype, D, bias)
    "2-odd-p": (2, (8, 9, 33, 100, 3, "bf16", "bf16", True, True)),
    "2-n7": (2, (100, 70, 5, 7, 7, "f32", "f32", True, True)),
    "2-n255": (2, (5, 13, 17, 255, 1, "bf16", "f32", False, True)),
    "2-n127": (2, (20, 12, 9, 127, 4, "f32", "f32", True, False)),
    "2-n4": (2, (32, 16, 130, 4, 2, "bf16", "bf16", True, True)),
    "2-one-row": (2, (64, 17, 1, 256, 1, "bf16", "bf16", True, True)),
    "4-odd-p": (4, (20, 15, 33, 100, 5, "bf16", "bf16", True, True)),
    "4-n255": (4, (40, 16, 7, 255, 2, "f32", "f32", True, True)),
    "4-n7": (4, (300, 100, 5, 7, 10, "bf16", "f32", True, True)),
    "4-n30": (4, (27, 21, 61, 30, 3, "bf16", "bf16", False, False)),
    "4-n129": (4, (100, 14, 3, 129, 7, "f32", "f32", True, True)),
    "4-n6": (4, (60, 20, 111, 6, 1, "bf16", "bf16", True, True)),
    "2-past-the-cache": (2, (64, 128, 33, 255, 8, "bf16", "f32", True, True)),
}
