"""The adapters' workspace size over calls of one server, on the CPU."""
import ctypes

import pytest

import w4a8_quantized_gemm_token_amd as w4

EWORKSPACE = 4


def parts(M, K, R):
    """Bytes that a slab of M rows uses: 64 bytes, a table entry of 32 bytes for each group that a tile of 64 rows can have and for
    its rows without one, and the low-rank values of each range of k: 512 units of tiles, four ranges at least, as far as there are
    eight windows of 64 k in each."""
    tiles, windows = -(-M // 64), -(-K // 64)
    splits = max(1, min(max(4, 512 // tiles), windows // 8))
    return 64 + tiles * (min(M, 64) + 1) * 32 + splits * M * R * 4


@pytest.mark.parametrize("K,R", [(8, 8), (1024, 16), (4096, 64), (8192, 128), (7168, 256), (1 << 20, 8)])
def test_never_falls_as_rows_grow(K, R):
    size = w4.load().w4a8_lora_workspace_size
    last = 0
    for M in sorted({*range(1, 9000), *range(9000, 33500, 7), 32767, 32768, 32769, 40000, 65536, (1 << 31) - 1}):
        need = size(M, K, 8, R)
        assert need >= last, f"M={M}: {need} bytes, a smaller batch {last}"
        # every slab of the call has room
        assert need >= parts(min(M, 32768), K, R)
        if M > 32768 and M % 32768:
            assert need >= parts(M % 32768, K, R)
        last = need


def test_never_falls_as_sizes_grow():
    size = w4.load().w4a8_lora_workspace_size
    for M in (1, 17, 64, 400, 2048, 5000, 40000):
        sizes = [size(M, K, 8, 16) for K in range(8, 20000, 8)]
        assert sizes == sorted(sizes)
        sizes = [size(M, 4096, 8, R) for R in range(8, 257, 8)]
        assert sizes == sorted(sizes)
        sizes = [size(M, 4096, L, 16) for L in (1, 2, 63, 64, 65, 1000, 65536)]
        assert sizes == sorted(sizes)


def test_one_byte_less_is_refused():
    lib = w4.load()
    f = ctypes.c_void_p(4096)
    for M, K, R in ((4, 256, 16), (2048, 8192, 128), (2049, 8192, 128), (5000, 8192, 128), (33000, 4096, 256)):
        need = lib.w4a8_lora_workspace_size(M, K, 8, R)
        args = [f, 0, K, M, K, f, f, f, 2, 8, R, None, None, f, 40, 40, f, 0, 40, f, need - 1, None]
        assert lib.w4a8_lora_add(*args) == EWORKSPACE
