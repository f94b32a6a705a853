"""The rule by which the product with epilogue is laid out (small_form and plan_tiles of rb_linear.hip), restated, so
that a test can say which of its forms a shape takes. The split's workspace ties it to the library's own rule."""

KINDS = {False: ((32, 0.79, 0.9), (64, 1.0, 1.15), (128, 1.07, 1.3)),
         True: ((32, 0.36, 0.38), (64, 0.50, 0.65), (128, 0.65, 0.95))}


def ceil(a, b):
    return -(-a // b)


def small_tiles(M, N, K, aligned):
    """(estimate, tile height, chunks)"""
    steps, best = ceil(K, 64), None
    for bm, one, every in KINDS[aligned]:
        tiles, c = ceil(M, bm) * ceil(N, 256), 1
        while c <= 16 and (c == 1 or (c * 2 <= steps and tiles * c <= 512)):
            blocks, each = tiles * c, ceil(steps, c)
            est = 5 + ceil(blocks, 256) * (each + 2) * (one + (every - one) * min(1.0, blocks / 256))
            est += 2 + c * M * N * 8 / 5e6 if c > 1 else 0
            if best is None or est < best[0]:
                best = est, bm, ceil(K, each * 64)
            c *= 2
    return best


def tiles(M, N, K, aligned):
    """(estimate, weight rows in 256-row tiles, tile height and chunks of the others)"""
    small, tm = small_tiles(M, N, K, aligned), ceil(M, 256)
    rounds = tm * ceil(N, 256) // 256
    if not aligned or rounds == 0:
        return small[0], 0, *small[1:]
    big = min(rounds * 256 // tm * 256, N)
    rest = small_tiles(M, N - big, K, aligned) if big < N else (0, 0, 0)
    est = rest[0] + 5 + rounds * (ceil(K, 64) + 2) * 1.6
    return (small[0], 0, *small[1:]) if big == 0 or small[0] < 0.87 * est else (est, big, *rest[1:])


def form(M, N, K, aligned):
    """"rows", "few", or tiles by their heights, + "join" where the columns are split."""
    est, big, bm, chunks = tiles(M, N, K, aligned)
    if K >= 8 and M <= 256:
        if M <= 4:
            return "rows"
        if 2.6 + ceil(ceil(N, 16) * ceil(M, 16), 256) * ceil(K, 64) * (0.13 if aligned else 0.33) < est:
            return "few"
    return "+".join(["256"] * (big > 0) + [str(bm)] * (big < N) + ["join"] * (chunks > 1))


def workspace(M, N, K):
    """Bytes of the partial sums, of whichever alignment needs more."""
    most = 0
    for aligned in (False, True):
        if form(M, N, K, aligned) not in ("rows", "few"):
            _, big, _, chunks = tiles(M, N, K, aligned)
            most = max(most, chunks * M * (N - big) * 4 if chunks > 1 else 0)
    return most
