"""A copy on the host of the rule by which tp_qgemm_fp8 picks its tile and the
splits of k, so that a test can say which one it reaches; and what its sums may
lose."""

CUS = 256
# What the 8-bit matrix instruction's sums of a block lose, at most, of the norm of
# the sums, as the contract states it.
LOST_8BIT = 5e-5


def plan(m, n, k, bf16):
    """(tile, splits of k): "few", (256, 256), (128, 128) or (64, 128)."""
    kb = k // 128
    tiles = lambda bm, bn: -(-m // bm) * -(-n // bn)  # noqa: E731
    rounds = lambda t: -(-t // CUS)  # noqa: E731
    if m <= 16 or (m <= 64 and -(-m // 16) * n * k <= 2 ** 25):
        return "few", 1
    step64, one128, two128 = (0.42, 0.72, 1.13) if bf16 else (0.8, 1.4, 2.8)
    r = rounds(tiles(128, 128))
    best, least = ((128, 128), 1), (r // 2 * two128 + r % 2 * one128) * kb
    big = rounds(tiles(256, 256)) * 2.05 * kb
    if bf16 and big < least:
        best, least = ((256, 256), 1), big
    t64, s = tiles(64, 128), 1
    while s <= kb and s <= 16 and (s == 1 or t64 * s <= CUS):
        sps = -(-kb // s)
        splits = -(-kb // sps)
        t = rounds(t64 * splits) * sps * step64 + (0.0 if splits == 1 else 3.0 + splits * m * n * 8.0 / 3e6)
        if t < least:
            best, least = ((64, 128), splits), t
        s += 1
    return best
