"""4-bit pages in plain torch: rows to codes and scales, and back in 64 bits."""

import torch

D = 256
BLOCK = 2304
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# scale bytes below 0xF8: bits 14..7 of an fp16
SCALES = torch.tensor([m * 2.0 ** -17 for m in range(8)] +
                      [(8 + m) * 2.0 ** (e - 18) for e in range(1, 31) for m in range(8)], dtype=torch.float64)
MOST = 0xE2  # 10240


def _nearest(x, table):
    """Index of the value of an ascending table nearest to x, the even one of two."""
    table = table.to(x.device)
    i = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
    down, up = x - table[i - 1], table[i] - x
    take_up = (up < down) | ((up == down) & (i % 2 == 0))
    return torch.where(take_up, i, i - 1)


def _f32(x):
    return x.float().double()


def quantize(x):
    """x [.., 256] (any float type): nibbles [.., 256] and scale bytes [.., 16], int64."""
    y = x.double().unflatten(-1, (16, 16))
    fine = torch.isfinite(y).all(-1)
    m = torch.where(fine, y.abs().amax(-1), 0.0)
    b = _nearest(_f32(m / 6.0), SCALES).clamp(max=MOST)
    s = SCALES.to(x.device)[b]
    q = torch.where((b > 0) & fine, 1.0 / s, 0.0)[..., None]
    q = torch.where(q > 0, _f32(y / s.clamp(min=2.0 ** -17)[..., None]), 0.0)
    code = _nearest(q.abs(), LEVELS) + 8 * (torch.signbit(q)).long()
    return code.flatten(-2), torch.where(fine, b, 0xFF)


def values(code, scale):
    """What nibbles and scale bytes stand for, in 64 bits (NaN for a scale byte of 0xFF)."""
    mag = LEVELS.to(code.device)[code & 7]
    v = torch.where(code > 7, -mag, mag).unflatten(-1, (16, 16))
    s = torch.cat([SCALES, torch.full((16,), float("nan"), dtype=torch.float64)]).to(code.device)[scale]
    return (v * s[..., None]).flatten(-2)


def turn(row):
    return (row & 1) | ((row // 4 % 4) << 1)


def _where(table, page, pos, n_kv):
    """(page, block, head, byte) of the codes' bytes [n, n_kv, 128] and the scales' [n, n_kv, 16] of positions."""
    dev = table.device
    pg = table[pos // page].long()[:, None, None]
    blk, row = (pos % page // 16)[:, None, None], (pos % 16)[:, None, None]
    head = torch.arange(n_kv, device=dev)[None, :, None]
    i = torch.arange(128, device=dev)[None, None]
    codes = row * 128 + (((i // 16) ^ turn(row)) * 16 + i % 16)
    scales = 2048 + row * 16 + torch.arange(16, device=dev)[None, None]
    return (pg, blk, head, codes), (pg, blk, head, scales)


def write(pool, table, page, pos, code, scale):
    """Rows (nibbles [n, n_kv, 256], scales [n, n_kv, 16]) to positions [n] of the sequence with pages `table` [width]."""
    at, sat = _where(table, page, pos, code.shape[1])
    pool[at] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    pool[sat] = scale.to(torch.uint8)


def read(pool, table, page, pos, n_kv):
    """(nibbles, scales) of positions."""
    at, sat = _where(table, page, pos, n_kv)
    b = pool[at].long()
    return torch.stack([b & 15, b >> 4], -1).flatten(-2), pool[sat].long()
