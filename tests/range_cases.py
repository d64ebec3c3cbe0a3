"""Shapes of the picks-only router gradient whose token ranges are long, and the
launches that they take: (T, d, N, k, lists' threads, ranges, whether a launch
of its own makes the pairs)."""
CASES = [
    (9001, 2048, 500, 4, 1024, 9, True),      # 1024-token ranges, the last of 809 tokens
    (9001, 2048, 500, 2, 256, 9, False),
    (5003, 2048, 500, 7, 1024, 10, True),     # 512
    (5003, 1024, 512, 16, 1024, 20, True),    # 256
    (1499, 2048, 500, 20, 1024, 12, True),    # 128, a wave per token's pairs
    (4500, 2048, 700, 4, 256, 5, True),       # more experts: four waves list
    (3001, 512, 4096, 8, 256, 3, True),
    (2100, 64, 4096, 64, 256, 3, True),
    (12345, 64, 2000, 1, 256, 13, False),
]
