"""Sizes of the feed-forward block's GPU tests that reach kernels by their plan
(test_ffn_plan.py checks on the CPU that every form a plan can choose is reached
by these and by the list in test_gpu_layer.py).

(M, H, F, group, activation, output type)"""

CASES = [
    # one or two rows, quantised by the down product's workgroups: one tile, two
    # tiles (from H = 5120 on), K-tiles that are no multiple of waves x stages
    (2, 128, 256, 64, "gelu", "f16"),
    (1, 5120, 128, 128, "silu", "bf16"),
    (2, 5120, 384, 64, "silu", "f16"),
    (1, 5120, 896, 64, "gelu", "bf16"),
    (1, 8192, 2688, 64, "silu", "f16"),
    (2, 8192, 2688, 128, "silu", "bf16"),
    (1, 8192, 4224, 128, "silu", "bf16"),
    (2, 5120, 4224, 64, "gelu", "f16"),
    # (their group parameters do not fit in LDS)
    (2, 5120, 28800, 64, "silu", "f16"),
    # few rows, streamed: one, two and four tiles, one and two row blocks, one to
    # eight waves
    (3, 128, 128, 64, "silu", "bf16"),
    (3, 5120, 128, 64, "silu", "f16"),
    (4, 5120, 384, 128, "gelu", "bf16"),
    (5, 5120, 640, 64, "silu", "f16"),
    (3, 10240, 256, 128, "silu", "f16"),
    (7, 10240, 640, 64, "silu", "bf16"),
    (9, 10240, 1152, 128, "gelu", "f16"),
    (17, 128, 128, 64, "gelu", "bf16"),
    (17, 2560, 128, 64, "silu", "f16"),
    (18, 2560, 256, 128, "silu", "bf16"),
    (20, 2560, 640, 64, "gelu", "f16"),
    (29, 2560, 1152, 128, "silu", "f16"),
    (33, 128, 128, 64, "silu", "f16"),
    (33, 256, 7168, 64, "gelu", "bf16"),
    (17, 10240, 128, 128, "silu", "bf16"),
    (19, 10240, 384, 64, "silu", "f16"),
    (23, 10240, 512, 128, "gelu", "bf16"),
    (31, 10240, 1152, 64, "silu", "f16"),
    # gate and up of four tiles and one row block, K over two, four and eight waves
    (2, 256, 24576, 64, "silu", "f16"),
    (9, 640, 24576, 128, "gelu", "bf16"),
    (16, 1408, 24576, 64, "silu", "bf16"),
    (13, 1152, 24576, 128, "silu", "f16"),
    # gate and up on 256-row tiles
    (1000, 8320, 8192, 128, "silu", "bf16"),
    (1000, 8320, 8192, 64, "gelu", "f16"),
    # down: the GEMM's 32 x 32 kernel with its own epilogue, and three splits of the
    # 16 x 16 one
    (513, 6656, 8320, 128, "silu", "bf16"),
    (600, 6656, 8320, 64, "silu", "f16"),
    (513, 3840, 3200, 64, "gelu", "bf16"),
    (520, 3840, 3200, 128, "silu", "f16"),
]
