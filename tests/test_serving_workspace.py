"""The serving operators' workspace sizes without a GPU: a workspace made for the largest batch
serves every smaller one."""
import pytest

from test_serving_abi import lib  # noqa: F401  (the library fixture)


@pytest.mark.parametrize("d_col", [8, 512, 513, 1408, 4096, 11008, 28672, 65536])
@pytest.mark.parametrize("rank", [1, 4, 16, 17, 64, 200, 256])
def test_lora_size_never_falls_as_tokens_grow(lib, d_col, rank):  # noqa: F811
    size = lib.gptqs_linear_lora_workspace_size
    last = 0
    for n in list(range(1, 4097)) + [8192, 16384, 65535 * 64]:
        now = size(n, d_col, rank)
        tiles, most = -(-n // 16) * -(-rank // 16), min(64, -(-d_col // 512))
        splits = min(most, -(-512 // tiles))         # the shares the columns are split into
        assert now >= last and now >= 4 * splits * n * rank, n
        last = now


def test_moe_size_never_falls_as_tokens_grow(lib):  # noqa: F811
    size = lib.gptqs_moe_workspace_size
    for d, f, e, k in ((256, 128, 8, 2), (2048, 1408, 64, 8), (99, 51, 6, 2), (64, 32, 512, 32)):
        sizes = [size(n, d, f, e, k) for n in range(1, 257)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:]))
