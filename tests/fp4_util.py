"""The microscaled 4-bit format from its definition, in numpy and 64 bits."""
import numpy as np
import torch

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# The e4m3 numbers from 0 to 448 in order: what the codes 0 ... 126 stand for.
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])


def nearest(x, unit, grid):
    """The index of the grid value nearest to x / unit (both >= 0), ties to the
    even index.  Compared as x against middle * unit, which f64 holds exactly."""
    middles = (grid[1:] + grid[:-1]) / 2
    x, unit = np.asarray(x, dtype=np.float64), np.asarray(unit, dtype=np.float64)
    lo, hi = np.zeros(np.shape(x), dtype=np.int64), np.full(np.shape(x), len(middles), dtype=np.int64)
    while (lo < hi).any():  # the number of middles that x is past
        mid = (lo + hi) // 2
        m = middles[np.minimum(mid, len(middles) - 1)] * unit
        past = np.where(mid % 2 == 0, x > m, x >= m) & (lo < hi)
        hi = np.where((lo < hi) & ~past, mid, hi)
        lo = np.where(past, mid + 1, lo)
    return lo


def quantised(x, block):
    """(codes, block scale bytes, row scales or None) of an M x K array.  A row
    (blocks of 16) or block (of 32) that holds an infinity or a NaN has codes of 0
    and a NaN scale."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    lost = ~np.isfinite(x)
    lost = lost.any(axis=1, keepdims=True) if block == 16 else np.logical_or.reduceat(lost, np.arange(0, K, 32), axis=1) \
        if K else lost
    x = np.where(np.repeat(lost, K if block == 16 else 32, axis=1)[:, :K], 0.0, x)
    blocks = -(-K // block)
    full = np.zeros((M, blocks * block))
    full[:, :K] = x
    b = np.abs(full).reshape(M, blocks, block)
    top = b.max(axis=2) if K else np.zeros((M, 0))
    if block == 16:
        most = top.max(axis=1) if K else np.zeros(M)
        e = np.full(M, -126)
        for i in range(M):
            while most[i] > 2688.0 * 2.0 ** e[i]:
                e[i] += 1
        r = np.where(most > 0, 2.0 ** e.astype(np.float64), 0.0)
        unit = np.where(most > 0, r, 1.0)
        bytes_ = nearest(top, 6.0 * unit[:, None], E4M3)
        scale = E4M3[bytes_] * unit[:, None]
    else:
        r = None
        e = np.frexp(top)[1] - 1 - 2
        e = np.where(top > 0, np.maximum(e, -127), -127)
        bytes_ = e + 127
        scale = 2.0 ** e.astype(np.float64)
    code = nearest(b, np.where(scale > 0, scale, 1.0)[:, :, None], VALUES)
    code = np.where(scale[:, :, None] > 0, code, 0).reshape(M, -1)[:, :K]
    if block == 16:
        r = np.where(lost[:, 0] if K else False, np.nan, r)
    else:
        bytes_ = np.where(lost, 255, bytes_)
    return code + 8 * np.signbit(x) * (code > 0), bytes_, r


def scale_place(i, b, blocks):
    """The byte of row i's block b in a matrix's scale tiles."""
    cols = -(-blocks // 4)
    return ((i // 128) * cols + b // 4) * 512 + 16 * (i % 32) + 4 * (i % 128 // 32) + b % 4


def packed(codes, bytes_, junk=0xEE, pitch=None, offset=0):
    """Codes (M x K) and scale bytes (M x blocks) as (codes' bytes, tiles) on the
    CPU; what is not defined (rows that are not there, padding of pitches) is junk."""
    M, K = codes.shape
    width = -(-K // 2)
    even = np.zeros((M, 2 * width), dtype=np.uint8)
    even[:, :K] = codes
    pitch = pitch or max(16, -(-width // 16) * 16)
    buf = np.full(offset + M * pitch + 16, junk, dtype=np.uint8)
    rows = buf[offset:offset + M * pitch].reshape(M, pitch)
    rows[:, :width] = even[:, 0::2] | (even[:, 1::2] << 4)
    blocks = bytes_.shape[1]
    R, C = -(-M // 128), -(-blocks // 4)
    tiles = np.full(R * C * 512, 0xFF, dtype=np.uint8)  # (NaN in both types)
    i, b = np.meshgrid(np.arange(M), np.arange(4 * C), indexing="ij")
    tiles[scale_place(i, b, blocks)] = 0
    i, b = np.meshgrid(np.arange(M), np.arange(blocks), indexing="ij")
    tiles[scale_place(i, b, blocks)] = bytes_
    return buf, (M, width, pitch, offset), tiles.reshape(R, C, 512)


def on_gpu(b, codes, bytes_, scales, block, **kw):
    """The library's operand (2-D) of these codes."""
    buf, (M, width, pitch, offset), tiles = packed(codes, bytes_, **kw)
    dev = torch.from_numpy(buf).cuda()
    view = dev[offset:offset + M * pitch].view(M, pitch)[:, :width]
    return b.Fp4Rows(view, torch.from_numpy(tiles).cuda(), None if scales is None else torch.from_numpy(
        np.asarray(scales, dtype=np.float32)).cuda(), block)


def values(codes, bytes_, scales, block):
    """The numbers that codes and scales stand for, in f64."""
    M, K = codes.shape
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = E4M3[bytes_] if block == 16 else 2.0 ** (bytes_.astype(np.float64) - 127)
    v = v * np.repeat(s, block, axis=1)[:, :K]
    return v if scales is None else v * np.asarray(scales, dtype=np.float64)[:, None]


def unpacked(rows, K):
    """(codes, scale bytes) of a 2-D operand that the library wrote."""
    raw = rows.codes.cpu().numpy()
    M = raw.shape[0]
    codes = np.stack([raw & 15, raw >> 4], axis=2).reshape(M, 2 * raw.shape[1])
    blocks = -(-K // rows.block)
    flat = rows.block_scales.cpu().numpy().reshape(-1)
    i, b = np.meshgrid(np.arange(M), np.arange(-(-blocks // 4) * 4), indexing="ij")
    return codes, flat[scale_place(i, b, blocks)]
