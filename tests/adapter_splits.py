"""How the adapter kernels split their work (csrc/adapter.h), for tests that
have to reach a split: a copy that test_adapter_splits_host.py holds against
the header."""


def tiles(rows, adapters):
    return (rows + 31 * min(adapters + 1, rows)) // 32


def parts(tiles, columns, rank):
    """K parts of the shrink."""
    groups = max(1, (tiles + 1) // 2 if rank > 64 else tiles)
    resident = 256 if rank <= 16 else 520 if rank <= 32 or rank > 64 else 800
    return max(1, min(256 // groups, columns // 256, 16), min(resident // groups, columns // 2048))


def expand_chunk(tiles, columns, rank):
    """Tiles of an expand workgroup."""
    blocks = (columns + 511) // 512
    return 1 if rank <= 32 else max(1, min(rank // 12, (tiles * blocks + 1023) // 1024))


def gradient_chunk(tiles, rank, n_in, n_out):
    """Tiles of a weight-gradient workgroup."""
    blocks = (n_in + 511) // 512 + (n_out + 511) // 512
    chunks = max(1, (256 if rank > 64 else 512) // blocks)
    return max(1, (tiles + chunks - 1) // chunks)
