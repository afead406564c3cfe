"""The 8-bit floating point operators from their definition, in 64 bits on the CPU: e4m3 values
with one scale for each block of 128, products of ragged buckets, the SwiGLU FFN."""
import numpy as np
import torch

BLOCK = 128
FLOOR = 2.0 ** -100
# the 127 non-negative e4m3 numbers, by code: exponent field 0 counts steps of 2^-9
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                 for c in range(127)])
BORDERS = (E4M3[1:] + E4M3[:-1]) / 2


def blocks(n):
    return -(-n // BLOCK)


def to_codes(v):
    """e4m3 codes (uint8) of float64 numbers in [-448, 448]: nearest, ties to the even code."""
    a = np.abs(v)
    lo = np.searchsorted(BORDERS, a, side="left")    # a on a border: the lower number
    hi = np.searchsorted(BORDERS, a, side="right")   # ... the upper one
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    return (code | (np.signbit(v) << 7)).astype(np.uint8)


def code_values(codes):
    codes = np.asarray(codes)
    mag = codes & 0x7F
    v = np.where(mag == 127, np.nan, E4M3[np.minimum(mag, 126)])
    return np.where(codes >> 7, -v, v)


def quantize(parts):
    """(codes, scale) of blocks given as [..., entries] float64, one scale per leading index."""
    with np.errstate(invalid="ignore", over="ignore"):
        finite = np.isfinite(parts).all(-1)
        m = np.maximum(np.abs(np.where(finite[..., None], parts, 0)).max(-1), FLOOR)
        codes = to_codes(np.where(finite[..., None], 448 * parts / m[..., None], 0))
    codes = np.where(finite[..., None], codes, np.uint8(0x7F))
    scale = m.astype(np.float32) / np.float32(448)
    return codes, np.where(finite, scale, np.float32(np.nan))


def quantize_rows(x):
    x = x.double().numpy()
    rows, cols = x.shape
    padded = np.zeros((rows, blocks(cols) * BLOCK))
    padded[:, :cols] = x
    codes, scale = quantize(padded.reshape(rows, -1, BLOCK))
    return codes.reshape(rows, -1)[:, :cols], scale


def quantize_weights(w):
    w = w.double().numpy()
    E, N, K = w.shape
    nb, kb = blocks(N), blocks(K)
    padded = np.zeros((E, nb * BLOCK, kb * BLOCK))
    padded[:, :N, :K] = w
    parts = padded.reshape(E, nb, BLOCK, kb, BLOCK).transpose(0, 1, 3, 2, 4)
    codes, scale = quantize(parts.reshape(E, nb, kb, -1))
    codes = codes.reshape(E, nb, kb, BLOCK, BLOCK).transpose(0, 1, 3, 2, 4)
    return codes.reshape(E, nb * BLOCK, kb * BLOCK)[:, :N, :K], scale


def rows_value(q, s):
    """float64 numbers that quantised rows (torch e4m3 and fp32 tensors) stand for."""
    q, s = q.cpu().float().double(), s.cpu().double()
    return q * s.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def weight_value(q, s):
    """float64 numbers that one expert's quantised weight stands for."""
    q, s = q.cpu().float().double(), s.cpu().double()
    return q * s.repeat_interleave(BLOCK, 0)[:q.shape[0]].repeat_interleave(BLOCK, 1)[
        :, :q.shape[1]]


def product(a, w):
    """(a w^T, |a| |w|^T): the result and the sum of its terms' magnitudes."""
    return a @ w.T, a.abs() @ w.abs().T


# How far an fp32 sum of the kernel may be from the exact one, relative to the sum of its
# terms' magnitudes S.  Within a block of 128: 4 MMAs of 32 products each; a tensor core aligns
# the 32 products and the running sum to the largest of them and may drop what lies below
# 2^-24 of it, so an MMA is off by at most 33 x 2^-24 of that block's S.  Between blocks: two
# scale products and an FMA, each off by 2^-24, and one addition more for each block.
def sum_error(K):
    return (4 * 33 + 3 + blocks(K)) * 2.0 ** -24


BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2
E4M3_HALF_STEP = torch.finfo(torch.float8_e4m3fn).eps / 2
