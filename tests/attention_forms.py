"""Shapes for each form that the attention kernels have, and which kernels they
take: test_attention_forms_host.py pins them on the CPU, test_gpu_attention_edges.py
runs them."""

# N, Hq, Hkv, D: kernels of the forward pass, dq, dk and dv (waves; "s": work groups
# share the keys or queries). "+" before a kernel's columns: by tiles of 128 queries.
BF16 = {
    (330, 2, 1, 64): ("rows 64", "rows 64 s", "kv 64 4 s"),
    (320, 2, 1, 64): ("rows 64", "rows 64 s", "kv 64 4 s"),
    (330, 3, 1, 128): ("rows 128", "rows 128 s", "kv 128 4 s"),
    (707, 64, 64, 88): ("rows 96", "rows 96", "kv 96 4"),
    (1040, 64, 16, 64): ("tiles 64", "tiles 64", "kv 64 8"),
    (1056, 64, 16, 64): ("tiles 64", "tiles 64", "kv 64 8"),
    (800, 64, 64, 64): ("tiles 64", "tiles 64", "kv 64 4"),
    (801, 64, 64, 40): ("tiles 64", "tiles 64", "kv 64 4"),
    (833, 64, 32, 88): ("tiles 96", "tiles 96", "kv 96 4"),
    (900, 64, 64, 128): ("tiles 128", "tiles 128", "kv 128 4"),
    (1120, 48, 12, 104): ("tiles 128", "tiles 128", "kv 128 4"),
}
F32 = {
    (330, 2, 1, 64): ("rows 64", "rows 64 s", "kv 64 4 s"),
    (320, 2, 1, 64): ("rows 64", "rows 64 s", "kv 64 4 s"),
    (330, 3, 1, 128): ("rows 128", "rows 128 s", "kv 128 4 s"),
    (707, 64, 64, 88): ("rows 96", "rows 96", "kv 96 4"),
    (1040, 64, 16, 64): ("rows 64", "rows 64", "kv 64 4"),
    (833, 64, 32, 88): ("tiles 96", "tiles 96", "kv 96 4"),
    (900, 64, 64, 128): ("tiles 128", "tiles 128", "kv 128 4"),
    (1120, 48, 12, 104): ("tiles 128", "tiles 128", "kv 128 4"),
}
