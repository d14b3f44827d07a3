"""How the gated delta rule deals a call out (csrc/ssm_deltarule.hip: cut_of, heads_together), worked out here from the sizes, so
that a test can say which form it reaches; tests/test_deltarule_plan.py holds it to the library's workspace query."""

CHUNK = {"bf16": 64, "f32": 32}
FRAGMENTS = {"bf16": 6, "f32": 2}  # of an inverse, 512 floats each


def up(n, m):
    return -(-n // m) * m


def cut(b, L, H, Dk, Dv, dtype):
    """(segments, parts a segment, chunks a part, parts before the last segment): one segment where a sequence is not cut."""
    at_once = 256
    chunks, heads = -(-L // CHUNK[dtype]), b * H
    tiles = -(-Dv // 64)
    more = tiles + -(-up(Dk, 16) // 64)
    best, least = (1, 1, max(1, chunks), 0), float(-(-heads * tiles // at_once) * chunks)
    if heads * tiles >= at_once:
        return best
    for segs in range(2, min(64, chunks // 2) + 1):
        for parts in range(1, 5):
            pc = -(-chunks // (segs * parts))
            n = -(-chunks // (pc * parts))
            if n < 2:
                continue
            n_parts = (n - 1) * parts
            cost = (float(-(-heads * tiles * n // at_once) * pc * parts) + 0.75 * float(-(-heads * more * n_parts // at_once) * pc)
                    + (0.35 if Dk <= 64 else 1.0) * float(n_parts) + 3.0)
            if cost < least:
                least, best = cost, (n, parts, pc, n_parts)
    return best


def heads_together(b, L, H, G, dtype):
    """Heads of a group whose gradients one workgroup takes, one after the other."""
    chunks, share = -(-L // CHUNK[dtype]), H // G
    heads = share
    while heads > 1 and (share % heads or b * (H // heads) * chunks < 1024):
        heads -= 1
    return heads


def workspace(b, L, H, G, Dk, Dv, dtype, backward):
    chunks = b * H * -(-L // CHUNK[dtype])
    KP, VP = up(Dk, 16), up(Dv, 16)
    n_parts = cut(b, L, H, Dk, Dv, dtype)[3]
    tri = up(chunks * FRAGMENTS[dtype] * 2048, 256)
    total = tri + up(b * H * n_parts * KP * VP * 4, 256) + up(b * H * n_parts * KP * KP * 4, 256)
    if backward:
        total += tri + 2 * up(chunks * KP * VP * 4, 256) + 2 * up(chunks * CHUNK[dtype] * VP * 4, 256)
        sets = H // heads_together(b, L, H, G, dtype)
        if sets != G:
            total += 2 * up(b * L * sets * Dk * 4, 256)
    return total
