"""The distillation's workspace size against its parts, counted here: a flag a
row, 16 bytes for each part a row is cut into where the loss runs in parts, and
the logits at the entries and the label where loss and gradient run in parts."""
import pytest

import fsdp_sharded_optimizer_zero_amd as Z

BLOCKS = 2048       # parts that fill the GPU; fewer are cut smaller


def least_bytes(rows, vocab, k, vector):
    vectors = vocab // vector
    one_block = rows >= 128 or vectors <= 1024          # loss and gradient
    loss_one_block = one_block and vectors <= 4096
    parts = -(-vocab // (8 * 256 * vector))
    if rows * parts < BLOCKS:
        parts = -(-vocab // (2 * 256 * vector))
    return 4 * rows + (0 if loss_one_block else 16 * rows * parts) \
        + (0 if one_block else 4 * (k + 1) * rows)


@pytest.mark.parametrize("dtype,vector", [(Z.ZS_BF16, 8), (Z.ZS_F32, 4)])
@pytest.mark.parametrize("k", [0, 1, 64, 1024])
def test_distill_workspace_is_the_sum_of_its_parts(dtype, vector, k):
    sides = [v * vector + d for v in (512, 1024, 1025, 4096, 4097, 16384) for d in (-1, 0, 1)]
    for rows in (0, 1, 2, 100, 127, 128, 500, 8192, 1 << 20):
        for vocab in sides + [1, 50257, 128256, 151937, 262144]:
            n = Z.zs_distill_workspace_bytes(Z.make_distill(rows, vocab, k, logits_dtype=dtype))
            least = least_bytes(rows, vocab, k, vector)
            assert least <= n < least + 3 * 256 + 4 and n % 256 == 0
