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


def slot_of(bounds, R, length, piece):
    """Run, first row and end of the rows of slot `piece` (first >= end: none).
    Runs are the rows before the segments, the segments, the rows behind them;
    the search keeps the last of 64 probes that does not lie behind the slot."""
    at = [0, *(min(max(b, 0), R) for b in bounds), R]
    v, n = 0, len(at) - 1
    while n > 1:
        step = ceil(n, 64)
        lane = next(i for i in range(63, -1, -1) if i == 0 or (i * step < n and at[v + i * step] // length + v + i * step <= piece))
        v += lane * step
        n = min(step, n - lane * step)
    return v, at[v] + (piece - at[v] // length - v) * length, at[v + 1]
