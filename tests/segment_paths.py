"""Host model of the kernels that a call of the segment product runs: the
rules of csrc/segment.hip on sizes, element size and alignment, so that tests
can say which tile and which split of the rows they reach."""

UNITS = 256                                  # compute units


def ceil(a, b):
    return -(-a // b)


def direct(size, *widths):
    """Rows of whole 16-byte groups: operands are copied straight into LDS."""
    return all(w * size % 16 == 0 for w in widths)


def product_tile(R, I, O, size, transposed=False):
    """Tile of y (of dx if transposed) and its steps of the summed index."""
    out, summed = (I, O) if transposed else (O, I)
    large = size == 2 and direct(size, I, O) and ceil(R, 256) * ceil(out, 256) >= 2 * UNITS
    return 256 if large else 128, ceil(summed * size, 64)


def dw_shape(R, E, I, O, size, aligned=True):
    """dw: (tile, tiles of a segment, rows of a chunk or 0, most chunks)."""
    large = aligned and size == 2 and direct(size, I, O) and E * ceil(I, 256) * ceil(O, 256) >= 2 * UNITS
    tile = 256 if large else 128
    tiles = ceil(I, tile) * ceil(O, tile)
    if E * tiles >= 2 * UNITS or R <= 4096:
        return tile, tiles, 0, 0
    chunk = ceil(max(256, ceil(R, max(1, 2 * UNITS // tiles))), 32) * 32
    return tile, tiles, chunk, R // chunk + E
