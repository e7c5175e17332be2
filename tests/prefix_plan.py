"""How kv_prefix_attention_run cuts a call, from its sizes: the rule of
csrc/kv_prefix.hip written out plainly, with the number of parts of the prefix
by trying all.  Its workspace size has to be the library's, so a test that
means one of the plans can see that it gets it."""
import numpy as np

STEP, HEAD = 32, 4 * (4096 + 4)  # tokens of a step; bytes of a line's starts


def own_shape(D, rows):
    """(row tiles of a wave, waves that take different rows) of the requests' kernel."""
    if rows <= 16:
        return 1, 1
    if D == 256:
        return 1, 2 if rows <= 32 else 4
    return 2, 1 if rows <= 32 else 2 if rows <= 64 else 4


def up(n, to):
    return -(-n // to) * to


def plan(R, M, Hq, Hkv, D, max_q, max_len, max_prefix):
    """dict: kind ("line": one line with the prefix; "last": the requests'
    kernel joins; "cut": their own line, cut on every start; "even": in equal
    runs), starts, slots, shape, parts, joins, bytes."""
    G = Hq // Hkv
    rows, every, steps = min(max_q, M) * G, M * G, -(-max_prefix // STEP)
    NR, RS = own_shape(D, rows)
    one, wide = every <= 16, D <= 128
    pNR, pW = (1, 4 if every <= 64 else 8) if D == 256 else (1 if D == 128 and every <= 192 else 2, 4)
    RW = 16 * NR * RS
    PW = RW if one else 16 * pNR * pW
    groups, pgroups = -(-rows // RW), -(-every // PW)
    starts = Hkv * (min(R, M) * groups + pgroups) if one else R * Hkv * groups
    slots = 256 * (3 if NR == 1 and wide else 2)
    if one:
        slots = 256 if starts <= 64 else 512 if starts <= 128 else max(2 * starts, slots)
    aligned = one or starts <= 256
    slots *= 1 if aligned else 2
    part_slots, part_rows, head = slots + (0 if aligned else starts), 16 if one else min(rows, RW), HEAD
    # the prefix's parts
    pairs, fit = Hkv * pgroups, 256 * (3 if pNR == 1 and D == 128 else 8 // pW)
    waves = 8 if wide and (NR == 1 or starts <= 256) else 4
    split = waves // RS
    whole = not one and starts <= 1024 and (max_len <= 1024 or (NR == 1 and wide and starts >= 128 and max_len <= 4096))
    k = np.arange(1, max(min(max(steps // 3, 1), 4 * fit // pairs), 1) + 1, dtype=np.int64)
    cost = (-(-pairs * k // fit)).astype(float) * ((-(-steps // k)).astype(float) + 12.0) + (Hkv * every * k * D).astype(float) * 8.0 / 5e6
    fold = 2.0 + 2.0 * k.astype(float) / split
    last = whole & (fold < 28.0)
    best = int(np.argmin(cost + np.where(last, fold, 28.0)))
    parts, last = int(k[best]), bool(last[best])
    if last:
        slots, part_slots, head = starts, 0, 0
    places = 0 if one else pairs * parts
    bytes_ = (up(head + (0 if one else HEAD), 256) + up(part_slots * part_rows * (D + 2) * 4, 256)
              + up(places * min(every, PW) * (D + 2) * 4, 256))
    return dict(kind="line" if one else "last" if last else "cut" if aligned else "even", starts=starts, slots=slots, shape=(NR, RS),
                parts=parts, joins=R * max_q * Hq, bytes=bytes_)
