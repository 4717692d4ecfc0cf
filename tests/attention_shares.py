"""Shapes at which work groups share the keys' queries of dk and dv, and how many,
without and with a prefix: test_attention_shares_host.py pins them on the CPU,
test_gpu_attention_shares.py runs those of up to 1100 rows."""

from sample_grad_norms_amd import _lib

# dtype, lengths, Hq, Hkv, D: work groups without and with a prefix
SHARES = {
    (_lib.BF16, (1040,), 192, 12, 64): (1, 2),
    (_lib.BF16, (1040,), 192, 12, 104): (3, 2),
    (_lib.F32, (1024,), 96, 6, 128): (3, 2),
    (_lib.F32, (700, 340), 192, 6, 128): (3, 2),   # by the average length, 16 steps of each of 32 heads
    (_lib.BF16, (1023,), 208, 13, 64): (1, 3),     # 496 steps
    (_lib.F32, (700, 310), 192, 6, 128): (3, 3),   # 480 steps
    (_lib.BF16, (4096, 4096), 16, 4, 64): (1, 2),
    (_lib.BF16, (8192,), 16, 2, 128): (3, 2),
    (_lib.BF16, (2048, 2048), 32, 8, 64): (1, 3),
}
